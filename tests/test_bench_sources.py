"""Which changes of the sources drop a measured traffic figure (host only)."""
import json
import os

import pytest

import bench

HEADER = open(os.path.join(bench.ROOT, "include", "lora_mi355x.h")).read()
SETS = [bench.BGMV_SOURCES, bench.PLANNED_SOURCES, bench.DEVPLAN_SOURCES]


@pytest.mark.parametrize("files", SETS)
def test_other_entry_points_and_comments_keep_the_figures(files):
    want = bench.source_hash(files)
    assert want == bench.source_hash(files, HEADER)
    added = HEADER.replace("#ifdef __cplusplus", """/* more calls */
#define LORA_NEW_LIMIT 7
typedef struct { int32_t a; const void* b; } lora_new_desc;
lora_status lora_new_call(const lora_pool* pool, const lora_new_desc* d, void* stream);
#ifdef __cplusplus""", 1)
    assert added != HEADER and bench.source_hash(files, added) == want
    assert bench.source_hash(files, HEADER.replace("bad argument", "a bad argument")) == want


@pytest.mark.parametrize("files,old,new", [
    *[(f, "LORA_BF16 = 2", "LORA_BF16 = 4") for f in SETS], *[(f, "#define LORA_MAX_IO 8", "#define LORA_MAX_IO 9") for f in SETS],
    (bench.PLANNED_SOURCES, "int32_t x_group;", "int64_t x_group;")])
def test_what_the_kernels_use_drops_them(files, old, new):
    assert old in HEADER
    assert bench.source_hash(files, HEADER.replace(old, new)) != bench.source_hash(files)


def test_the_headline_has_its_figure():
    # of the kernels as they are; a change of them needs the counters taken again
    records = json.load(open(os.path.join(bench.ROOT, "profiles", "hbm_traffic.json")))["records"]
    taken = {r["kernel_source_hash"] for r in records.values()}
    for files in SETS:
        if bench.source_hash(files) not in taken:
            pytest.skip("the kernels have changed since")
    got = bench.measured_traffic("llama7b_decode_bgmv", "lora_bgmv_apply", bench.source_hash(bench.BGMV_SOURCES))
    assert got == records["llama7b_decode_bgmv/lora_bgmv_apply"]["hbm_bytes_per_step"]
