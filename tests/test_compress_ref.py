"""The 64-bit definitions in compress_ref.py against definitions written
another way (exact fractions, scalar loops, torch's own 8-bit type), so that a
mistake in them cannot hide behind its copies elsewhere."""
import math
import random
from fractions import Fraction

import pytest
import torch

import compress_ref as ref


def e4m3_table():
    """Code to value through torch's 8-bit type."""
    return torch.arange(256, dtype=torch.int16).to(torch.uint8).view(torch.float8_e4m3fn).double().tolist()


def test_every_e4m3_code():
    ours = ref.values(torch.arange(256, dtype=torch.int16).to(torch.uint8), "e4m3").tolist()
    for a, b in zip(ours, e4m3_table()):
        assert (math.isnan(a) and math.isnan(b)) or a == b
    assert sum(math.isnan(x) for x in ours) == 2 and max(x for x in ours if x == x) == 448.0


def test_every_int8_code():
    got = ref.values(torch.arange(256, dtype=torch.int16).to(torch.uint8), "int8").tolist()
    assert got == [int.from_bytes(bytes([c]), "little", signed=True) for c in range(256)]


def test_rounding_between_every_pair_of_e4m3_values():
    """The midpoint goes to the even code, anything off it to the nearer value."""
    table = e4m3_table()[:127]
    for c in range(126):
        lo, hi = table[c], table[c + 1]
        mid = (lo + hi) / 2
        even = lo if c % 2 == 0 else hi
        for x, want in ((lo, lo), (mid, even), (math.nextafter(mid, 0.0), lo), (math.nextafter(mid, 1e9), hi), (hi, hi)):
            for sign in (1.0, -1.0):
                got = ref.nearest(torch.tensor([sign * x], dtype=torch.float64), "e4m3")
                assert float(got[0]) == sign * want
                assert ref.values(ref.codes_of(got, "e4m3"), "e4m3").tolist() == got.tolist()
    assert ref.nearest(torch.tensor([1e4, -1e4], dtype=torch.float64), "e4m3").tolist() == [448.0, -448.0]


def test_rounding_to_int8():
    rng = random.Random(1)
    xs = [i / 2 for i in range(-260, 261)] + [rng.uniform(-130, 130) for _ in range(500)]
    got = ref.nearest(torch.tensor(xs, dtype=torch.float64), "int8")
    assert got.tolist() == [max(-127, min(127, round(Fraction(x)))) for x in xs]     # Fraction rounds half to even
    assert ref.values(ref.codes_of(got, "int8"), "int8").tolist() == got.tolist()


def eight_bits(x):
    """Whether x = n * 2^e with n below 2^8."""
    m, _ = math.frexp(float(x))
    return m * 256 == int(m * 256)


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_scales_are_the_least_with_eight_bits(kv):
    rng = random.Random(2)
    values = [448.0, 127.0, 1.0, 3.0, 0.875, 2.0 ** -133, 3 * 2.0 ** -133, 3.3895313892515355e38]
    values += [float(torch.tensor(math.exp(rng.uniform(-80, 80))).to(torch.bfloat16)) for _ in range(300)]
    for a in values:
        s = float(ref.block_scale(torch.tensor(a), kv))
        assert eight_bits(s)
        q = Fraction(a) / int(ref.RANGE[kv])
        m, e = math.frexp(s)
        below = Fraction(m) - Fraction(1, 256) if m > 0.5 else Fraction(m) - Fraction(1, 512)   # the number before s
        assert Fraction(s) >= q > below * Fraction(2) ** e
    assert float(ref.block_scale(torch.tensor(0.0), kv)) == 0.0


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_append_element_by_element(kv):
    """Scalars and exact fractions, nearest code by search over all of them."""
    codes = [x for x in (e4m3_table() if kv == "e4m3" else range(-127, 128)) if x == x]
    codes = sorted({float(x) for x in codes})

    def nearest(x):
        best = min(abs(Fraction(c) - x) for c in codes)
        near = [c for c in codes if abs(Fraction(c) - x) == best]
        if len(near) == 1:
            return near[0]
        if kv == "int8":
            return next(c for c in near if int(c) % 2 == 0)
        return next(c for c in near if int(ref.codes_of(torch.tensor([c], dtype=torch.float64), kv)[0]) % 2 == 0)

    g = torch.Generator().manual_seed(3)
    B, Hkv, L, D, T = 2, 1, 40, 2, 16
    vals = torch.zeros((B, Hkv, L, D), dtype=torch.float64)
    scale = torch.full((B, Hkv, 3), 7.0, dtype=torch.float64)
    mine, mine_s = vals.clone(), scale.clone()
    end = [0, 0]
    for n, grow, news in ((20, 1.0, [20, 5]), (7, 3.0, [7, 7]), (1, 9.0, [1, 0]), (30, 0.1, [30, 9])):
        new = (torch.randn((B, n, Hkv, D), generator=g) * grow).to(torch.bfloat16)
        end = [e + m for e, m in zip(end, news)]
        ref.append(vals, scale, new, end, news, T, kv)
        for b in range(B):
            start = end[b] - news[b]
            for blk in range(3):
                inside = [t for t in range(blk * T, min(blk * T + T, L)) if start <= t < end[b]]
                if not inside:
                    continue
                top = max(abs(float(new[b, t - start, 0, d])) for t in inside for d in range(D))
                s, old = float(ref.block_scale(torch.tensor(top), kv)), float(mine_s[b, 0, blk])
                older = range(blk * T, max(start, blk * T)) if start > blk * T else []
                if len(older):
                    s = max(s, old)
                    if s > old:
                        for t in older:
                            for d in range(D):
                                mine[b, 0, t, d] = nearest(Fraction(float(mine[b, 0, t, d])) * Fraction(old) / Fraction(s))
                mine_s[b, 0, blk] = s
                for t in inside:
                    for d in range(D):
                        mine[b, 0, t, d] = nearest(Fraction(float(new[b, t - start, 0, d])) / Fraction(s))
        assert torch.equal(mine, vals) and torch.equal(mine_s, scale)


def test_attention_by_scalars():
    g = torch.Generator().manual_seed(4)
    B, q_len, Hq, Hkv, L, D = 2, 3, 4, 2, 6, 5
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((B, q_len, Hq, D), (B, Hkv, L, D), (B, Hkv, L, D)))
    lens = [6, 2]
    out, lse, w, _ = ref.attention(q, k, v, lens, 0.3)
    total = torch.zeros(B, Hkv, L, dtype=torch.float64)
    for b in range(B):
        for j in range(q_len):
            sees = lens[b] - (q_len - 1 - j)
            for i in range(Hq):
                h = i * Hkv // Hq
                if sees < 1:
                    assert torch.all(out[b, j, i] == 0) and lse[b, j, i] == -math.inf
                    continue
                e = [math.exp(0.3 * sum(float(q[b, j, i, d] * k[b, h, t, d]) for d in range(D))) for t in range(sees)]
                assert math.isclose(float(lse[b, j, i]), math.log(sum(e)), rel_tol=1e-12, abs_tol=1e-12)
                for t in range(sees):
                    total[b, h, t] += e[t] / sum(e)
                for d in range(D):
                    want = sum(e[t] * float(v[b, h, t, d]) for t in range(sees)) / sum(e)
                    assert math.isclose(float(out[b, j, i, d]), want, rel_tol=1e-11, abs_tol=1e-12)
    assert torch.allclose(w, total, rtol=1e-11, atol=1e-13)


def test_evict_by_repeated_choice():
    rng = random.Random(5)
    for _ in range(300):
        n, keep = rng.randint(1, 12), rng.randint(1, 12)
        recent = rng.randint(0, keep)
        w = [rng.choice([0.0, -0.0, 1.0, 2.0, math.nan, math.inf, -math.inf, -1.0]) for _ in range(n)]
        if n <= keep:
            want = list(range(n))
        else:
            left = list(range(n - recent))
            chosen = list(range(n - recent, n))
            for _ in range(keep - recent):
                best = left[0]
                for t in left[1:]:
                    if w[t] > w[best] or (math.isnan(w[best]) and not math.isnan(w[t])):
                        best = t
                left.remove(best)
                chosen.append(best)
            want = sorted(chosen)
        assert ref.evict(w, n, keep, recent) == want
