"""The cases of kv_cases.py reach every kernel variant that is built and every plan: the choice is the
host plan's, so a threshold that moves cannot drop a path from the GPU tests unseen (no GPU needed)."""
import kv_cases
import kv_plan


def variants_of(c):
    """(kernel size, exact, dtype, tile, 16-row tiles, waves) of the call's launches."""
    p = kv_plan.plan(*kv_cases.sizes(c))
    size = 64 if c.hd <= 64 else 128 if c.hd <= 128 else 256
    return p, {(size, c.hd == size, c.dtype, r.tile, r.nt, r.waves) for r in (p.prefix, p.own) if r.slots}


def built():
    """What launch_rows has: every (16-row tiles, waves) by kernel, size and type."""
    out = set()
    for size in (64, 128, 256):
        for dtype in (kv_cases.BF16, kv_cases.FP32):
            wide, f32 = size == 256, dtype == kv_cases.FP32
            rows = [(1, 4)] + ([] if wide and f32 else [(2, 4)]) + ([] if wide or f32 else [(1, 8), (1, 16)])
            tile = [(1, 4)] + ([(1, 8)] if wide != f32 else [] if wide else [(2, 4), (2, 8)])
            for exact in (True, False):
                out |= {(size, exact, dtype, 0, *x) for x in rows} | {(size, exact, dtype, 1, *x) for x in tile}
    return out


def test_every_kernel_variant():
    seen = set()
    for c in kv_cases.cases():
        p, v = variants_of(c)
        assert p.fits
        seen |= v
    assert len(built()) == 56
    assert seen == built(), (built() - seen, seen - built())


def test_every_plan():
    """Per kernel size, whole or below it: pieces and whole contexts, prefixes in the same launch, in one of
    their own, first and alone, and the own tokens' workgroups finishing a prefix with each count of waves."""
    seen = set()
    for c in kv_cases.cases():
        p, v = variants_of(c)
        (size, exact, dtype, *_), = {x[:3] for x in v}
        ls = [l[0] for l in kv_plan.launches(*kv_cases.sizes(c))]
        how = ("own cut" if p.cut else "own whole" if p.own.slots else "no own",
               "lead" if p.lead else "none" if not p.prefix.slots else "finish %d" % p.own.waves if p.finish else
               "same launch" if ls[0] == 0 and 1 not in ls and p.own.slots else "apart")
        assert (kv_plan.JOIN in ls) == (not p.direct and not p.finish)
        seen.add((size, exact, dtype) + how)
    for size in (64, 128, 256):
        for exact in (True, False):
            for dtype in (kv_cases.BF16, kv_cases.FP32):
                want = {("own cut", "none"), ("own whole", "none"), ("own whole", "same launch"), ("own cut", "same launch"),
                        ("own cut", "apart"), ("own whole", "lead"), ("no own", "apart")}
                if size < 256 and dtype == kv_cases.BF16:
                    want |= {("own whole", f"finish {w}") for w in (4, 8, 16)}
                missing = {w for w in want if (size, exact, dtype) + w not in seen}
                assert not missing, (size, exact, dtype, missing, sorted(x[3:] for x in seen if x[:3] == (size, exact, dtype)))
