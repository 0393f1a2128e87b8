"""Properties of the compiled tile kernel of the 8-bit product (no GPU needed).

It waits for its direct global->LDS loads by count, and after a whole tile may leave that tile's stores outstanding as
well.  An operation more makes such a wait stricter; one less would let a load that is needed be in flight: a tile's way
out past the cache must be as many stores as the wait assumes, and what was taken to be a step's loads must be there.
Nothing may spill, and no accumulator be moved between the multiplications."""
import re

import pytest

from test_kernel_asm import _device_asm

# tile and waves: (TC, TR, loads of a half); a wave stores 2 TC elements a lane, two of TR x 16 rows at a time
TILES = {"ILi256ELi256ELi2ELi4E": (4, 2, 4), "ILi128ELi128ELi2ELi2E": (2, 2, 4)}


@pytest.fixture(scope="module")
def bodies(tmp_path_factory):
    asm = _device_asm(tmp_path_factory, "fp8_product.hip")
    found = {}
    for m in re.finditer(r"^(_ZN4mssm12_GLOBAL__N_119(?:tile|fine)_product_kernel\S+):.*?^\.Lfunc_end", asm, re.M | re.S):
        found[m.group(1)] = m.group(0).split("\n")
    return asm, found


def test_every_instantiation_is_there_and_none_spills(bodies):
    asm, found = bodies
    # tiles of 256 x 256 and 128 x 128, with bf16 and with fp32 results, each with either kind of scales
    assert len(found) == 8, sorted(found)
    for name in found:
        md = asm[asm.index(".name:           " + name):]
        assert int(re.search(r"\.vgpr_spill_count:\s+(\d+)", md).group(1)) == 0, name
        assert int(re.search(r"\.private_segment_fixed_size:\s+(\d+)", md).group(1)) == 0, name


def test_loads_and_stores_are_those_that_the_waits_count(bodies):
    _, found = bodies
    for name, body in found.items():
        if "fine" in name:
            continue
        tile = next(t for t in TILES if t in name)
        tc, tr, loads = TILES[tile]
        at = [i for i, ln in enumerate(body) if "v_mfma_" in ln]
        loop = body[at[0]:at[-1] + 1]
        first = next(i for i in range(at[0], 0, -1) if "Loop Header: Depth=2" in body[i])
        end = next(i for i in range(at[-1], len(body)) if "s_barrier" in body[i])
        step = body[first:end]
        assert sum("global_load_lds_dwordx4" in ln for ln in step) == 2 * loads, name
        assert sum(bool(re.search(r"global_load_lds_(dword|ushort|ubyte) ", ln)) for ln in step) == 2, name
        others = [ln for ln in step if re.match(r"\s+(global_|buffer_|scratch_|flat_)", ln) and "global_load_lds" not in ln]
        assert not others, (name, others[:3])
        assert not [ln for ln in loop if "accvgpr" in ln], name
        waits = {int(v) for ln in body for v in re.findall(r"vmcnt\((\d+)\) lgkmcnt\(0\)", ln)}
        ahead = 2 * loads + 2
        stores = tr * 16 // 2
        assert {ahead, ahead + stores} <= waits, (name, waits)
        assert sum(bool(re.search(r"global_store_.* nt$", ln)) for ln in body) == stores, name
        assert sum(f"global_store_dwordx{tc}" in ln and " nt" in ln for ln in body) == stores, name
