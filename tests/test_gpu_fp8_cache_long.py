"""The paged cache's calls at lengths where a CTA takes several rows or tokens: reads above 2368 rows (16
CTAs per SM of one row), cu_rows too many to stage (above 511 sequences), writes of several strips of
columns with the four-load walk."""
import pytest
import torch

import bit_diffusion_transformer_b200 as opq
import fp8_reference as ref
from test_gpu_fp8 import F8, make_cache, no_device_error, randn, same_codes, same_scales  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"


def expected(cpu, i, slots, dtype):
    """code x scale of the given flat slots: rounded to fp32, then to the output's type."""
    c, s = cpu[2 * i], cpu[2 * i + 1]
    H, D = c.shape[2:]
    v = c.view(torch.uint8).reshape(-1, H, D)[slots].view(F8).double()
    s = s.reshape(-1, H, s.shape[3])[slots].double().repeat_interleave(128, 2)[..., :D]
    return (v * s).float().to(dtype)


def plan_read(lens, starts, page, gaps, seed):
    """A page table, cu_rows, the slot of every row (-1: of no sequence) and the pages needed."""
    need = [-(-(st + n) // page) for n, st in zip(lens, starts)]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    table = torch.full((len(lens), max(max(need), 1) + 1), -7, dtype=torch.int32)
    cu, slots, at = [gaps[0]], [-1] * gaps[0], 0
    for b, (n, st) in enumerate(zip(lens, starts)):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        pos = torch.arange(st, st + n)
        slots += (table[b].long()[pos // page] * page + pos % page).tolist()
        cu.append(cu[-1] + n)
    slots += [-1] * gaps[1]
    return table, torch.tensor(cu, dtype=torch.int32), torch.tensor(slots), pages


@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,heads,dims,page", [
    ([1700, 0, 1, 2313, 640, 346], 2, (64, 128), 16),         # 5000 rows: three a CTA
    ([9000, 33], 3, (80, 48), 7),                             # four
    ([2500, 2600], 30, (128, 128), 64),                       # wide rows: the chunks go round the threads
    ([20000, 20001], 1, (16, 32), 128),                       # 17, 64 threads a row
    ([151000], 1, (16, 16), 128)])                            # 64 rows, the most a CTA takes
def test_long_read(lens, heads, dims, page, dtype, layout):
    starts = [(5 * b + 3) % 11 for b in range(len(lens))]
    table, cu, slots, pages = plan_read(lens, starts, page, (2, 5), seed=len(lens))
    cpu, dev = make_cache(pages, page, heads, dims, layout, seed=7)
    live = slots >= 0
    out = [torch.full((len(slots), heads, D), 7.0, dtype=dtype, device=DEV) for D in dims]
    opq.fp8_cache_read(dev, table.to(DEV), cu.to(DEV), starts=torch.tensor(starts, dtype=torch.int32, device=DEV), out=out)
    for i, g in enumerate(out):
        assert torch.equal(g[live.to(DEV)].cpu(), expected(cpu, i, slots[live], dtype))
        assert bool((g[~live.to(DEV)] == 7.0).all())          # rows of no sequence stay


@pytest.mark.parametrize("seqs", [511, 512, 600, 2001])
def test_read_of_many_sequences(seqs):
    lens = [(7 * b) % 13 for b in range(seqs)]
    starts = [b % 5 for b in range(seqs)]
    table, cu, slots, pages = plan_read(lens, starts, 8, (0, 0), seed=seqs)
    cpu, dev = make_cache(pages, 8, 2, (64, 64), seed=3)
    got = opq.fp8_cache_read(dev, table.to(DEV), cu.to(DEV), len(slots),
                             starts=torch.tensor(starts, dtype=torch.int32, device=DEV))
    for i, g in enumerate(got):
        assert torch.equal(g.cpu(), expected(cpu, i, slots, torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,heads,dims,page", [
    (2000, 30, (128, 128), 64),      # 60 columns: four strips of 16 groups
    (2000, 30, (192, 128), 64),      # 90, two blocks a head on one side
    (1999, 30, (64, 32), 16),        # narrow heads: 32 groups
    (700, 9, (576, 512), 24),
    (40000, 1, (16, 16), 128)])      # 64 tokens, the most a CTA takes
def test_long_write(T, heads, dims, page, dtype):
    pages = -(-T // page) + 2
    cpu, dev = make_cache(pages, page, heads, dims, seed=T)
    kv = [randn(T, heads, D, seed=D, dtype=dtype) for D in dims]
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(1))[:T].long()
    slots[5::97] = -1
    opq.fp8_cache_write(*[t.to(DEV) for t in kv], dev, slots.to(DEV))
    live = slots >= 0
    untouched = torch.ones(pages * page, dtype=torch.bool)
    untouched[slots[live]] = False
    for i, x in enumerate(kv):
        D, nb = x.shape[2], dev[2 * i + 1].shape[3]
        codes, scales = dev[2 * i].view(torch.uint8).view(-1, heads, D), dev[2 * i + 1].view(-1, heads, nb)
        for b in range(nb):
            part = slice(b * 128, min(D, b * 128 + 128))
            c, s = ref.block_codes(x[live][:, :, part].double())
            same_codes(codes[slots[live].to(DEV)][:, :, part].contiguous().view(F8), c)
            same_scales(scales[slots[live].to(DEV)][:, :, b], s)
        was, sw = cpu[2 * i].view(torch.uint8).view(-1, heads, D), cpu[2 * i + 1].view(-1, heads, nb)
        assert torch.equal(codes[untouched.to(DEV)].cpu(), was[untouched])
        assert torch.equal(scales[untouched.to(DEV)].cpu(), sw[untouched])
