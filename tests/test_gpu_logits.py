"""Logit rules (moe_q4_logits_apply) against a plain implementation.

Each step of the rules is one binary32 rounding, so the processed logits are
compared bit for bit with numpy's binary32 steps, and those with binary64 ones
(four roundings, each at most 2^-24 of the larger of what it reads and gives).
The greedy token follows from the bits.  log-sum-exp: each exponential within
2^-24 * (4 + 2 |l - max|) of its value (the function's argument is scaled by
log2 e in binary32), the sum's roundings at most 64 on the way of any term, the
logarithm and the last addition 2^-24 * (2 + |lse| + |max|) more; the mean of
|l - max| under the softmax is at most log(vocab).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import quantized_moe_q4_b200 as m  # noqa: E402

NEG = np.float32(-np.inf)


def make(seed, T, V, hist=0, bias=0, masks=0, generated=True, hot=False):
    """Host arrays of one call; absent parts are absent keys."""
    rng = np.random.default_rng(seed)
    d = {"logits": (rng.standard_normal((T, V)) * 3).astype(np.float32)}
    if hist:
        lens = rng.integers(0, 2 * hist + 1, T)
        lens[rng.integers(0, T)] = 0
        lens[T - 1] = hist
        d["row_start"] = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        tok = rng.random(int(lens.sum())) ** (20 if hot else 3) * V
        d["tokens"] = np.minimum(tok.astype(np.int32), V - 1)
        if generated:
            d["generated_start"] = (d["row_start"][:-1] + (rng.random(T) * (lens + 1)).astype(np.int64)).astype(np.int64)
        d["repetition"] = (1 + rng.random(T)).astype(np.float32)
        d["presence"] = rng.standard_normal(T).astype(np.float32)
        d["frequency"] = rng.standard_normal(T).astype(np.float32)
    if bias:
        k = min(bias, V)
        lens = np.where(rng.random(T) < 0.7, k, 0)
        lens[0] = k
        d["bias_start"] = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        d["bias_token"] = np.concatenate([rng.permutation(V)[:n] for n in lens]).astype(np.int32)
        v = (rng.standard_normal(len(d["bias_token"])) * 5).astype(np.float32)
        v[rng.random(len(v)) < 0.1] = NEG
        d["bias_value"] = v
    if masks:
        bits = rng.random((masks, (V + 31) // 32 * 32)) < rng.random((masks, 1))
        bits[-1] = False
        d["mask"] = np.packbits(bits, axis=1, bitorder="little").view(np.int32)
        d["mask_row"] = rng.integers(-1, masks, T).astype(np.int32)
        d["mask_row"][T - 1] = masks - 1   # a row whose mask leaves nothing
    return d


def plain(d, kind):
    """(processed logits, sum of the magnitudes that the roundings go by) with every step in `kind`."""
    l = d["logits"].astype(kind)
    size = np.abs(l).astype(np.float64)
    T, V = l.shape
    with np.errstate(all="ignore"):
        for t in range(T):
            if "row_start" in d:
                lo, hi = (int(np.clip(v, 0, len(d["tokens"]))) for v in d["row_start"][t:t + 2])
                mid = int(d["generated_start"][t]) if "generated_start" in d else lo
                tok, at = d["tokens"][lo:hi], np.arange(lo, max(lo, hi))
                ok = (tok >= 0) & (tok < V)
                seen = np.bincount(tok[ok], minlength=V) > 0
                c = np.bincount(tok[ok & (at >= mid)], minlength=V).astype(np.float32).astype(kind)
                rep, pres, freq = (kind(d[k][t]) if k in d else kind(w) for k, w in (("repetition", 1), ("presence", 0), ("frequency", 0)))
                l[t] = np.where(seen, np.where(l[t] > 0, l[t] / rep, l[t] * rep), l[t])
                size[t] += np.abs(l[t]) + np.abs(freq * c) + np.where(c > 0, abs(pres), 0)
                l[t] = np.where(c > 0, (l[t] - freq * c) - pres, l[t])
            if "bias_start" in d:
                lo, hi = (int(np.clip(v, 0, len(d["bias_token"]))) for v in d["bias_start"][t:t + 2])
                last = {int(v): i for i, v in zip(range(lo, hi), d["bias_token"][lo:hi]) if 0 <= v < V}
                for v, i in last.items():
                    l[t, v] = l[t, v] + kind(d["bias_value"][i])
                    size[t, v] += abs(float(d["bias_value"][i])) if np.isfinite(d["bias_value"][i]) else 0.0
            if "mask" in d:
                r = int(d["mask_row"][t]) if "mask_row" in d else t
                if r != -1:
                    bits = np.unpackbits(d["mask"][r].view(np.uint8), bitorder="little")[:V] if 0 <= r < len(d["mask"]) else np.zeros(V)
                    l[t] = np.where(bits > 0, l[t], kind(-np.inf))
    return l, size


def rules(d):
    return m.LogitRules(**{k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in d.items() if k != "logits"})


def apply(d, want=("out", "token", "lse"), logits=None, in_place=False):
    T, V = d["logits"].shape
    l = torch.from_numpy(d["logits"]).cuda() if logits is None else logits
    out = (l if in_place else torch.empty(T, V, device="cuda")) if "out" in want else None
    token = torch.full((T,), -7, dtype=torch.int32, device="cuda") if "token" in want else None
    lse = torch.full((T,), 7.0, device="cuda") if "lse" in want else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.moe_q4_logits_apply(rules(d), l, out=out, token=token, lse=lse, status=status)
    torch.cuda.synchronize()
    return [None if v is None else v.cpu().numpy() for v in (out, token, lse)] + [int(status)]


def check(d, got):
    out, token, lse = got[:3]
    ref, _ = plain(d, np.float32)
    ref64, size = plain(d, np.float64)
    T, V = ref.shape
    if out is not None:
        assert np.array_equal(out, ref, equal_nan=True)
        fine = np.isfinite(ref64)
        assert np.array_equal(fine, np.isfinite(out))
        assert np.all(np.abs(out[fine] - ref64[fine]) <= 4 * 2.0 ** -24 * size[fine])
    key = np.where(np.isnan(ref), NEG, ref)
    top = key.max(1)
    if token is not None:
        assert np.array_equal(token, np.where(top == NEG, -1, key.argmax(1)))
    if lse is not None:
        for t in range(T):
            if np.isnan(ref[t]).any():
                assert np.isnan(lse[t])
            elif not np.isfinite(top[t]):
                assert lse[t] == top[t]
            else:
                e = ref[t].astype(np.float64)
                want = float(top[t]) + np.log(np.exp(e - float(top[t])).sum())
                tol = 2.0 ** -24 * (4 + 2 * np.log(V) + 64 + 2 + abs(want) + abs(float(top[t])))
                assert abs(float(lse[t]) - want) <= tol, (t, lse[t], want)


@pytest.mark.parametrize("T,V,hist,bias,masks", [
    (1, 131072, 1000, 0, 0), (1, 1, 0, 0, 0), (1, 1, 3, 1, 1), (2, 31, 5, 4, 2), (3, 33, 40, 33, 2), (5, 1000, 0, 0, 0),
    (4, 1025, 0, 20, 0), (4, 4099, 0, 0, 3), (33, 32003, 100, 300, 3), (7, 131072, 3000, 64, 4), (2, 151936, 500, 10, 2),
    (2, 300001, 700, 30, 2), (160, 5000, 30, 5, 8), (600, 513, 20, 3, 4), (1300, 64, 9, 3, 3), (2, 65536, 0, 0, 1)])
def test_rules_match_the_plain_steps(T, V, hist, bias, masks):
    d = make(T + V, T, V, hist, bias, masks)
    got = apply(d)
    check(d, got)
    assert got[3] == 0
    # each output alone, and in place, gives the same bits
    for want in (("out",), ("token",), ("lse",)):
        alone = apply(d, want)
        for a, b in zip(alone[:3], got[:3]):
            assert a is None or np.array_equal(a, b)
    there = apply(d, in_place=True)
    assert all(np.array_equal(a, b) for a, b in zip(there[:3], got[:3]))


def test_parts_alone_and_neutral_values():
    d = make(1, 6, 3001, 200, 10, 2)
    for keys in (("tokens", "row_start", "repetition"), ("tokens", "row_start", "frequency"),
                 ("tokens", "row_start", "generated_start", "presence"), ("tokens", "row_start"),
                 ("bias_token", "bias_value", "bias_start"), ("mask", "mask_row"), ("presence", "frequency")):
        part = {k: d[k] for k in ("logits",) + keys}
        check(part, apply(part))
    # nothing at all: a copy
    part = {"logits": d["logits"]}
    assert np.array_equal(apply(part, ("out",))[0], d["logits"])


def test_counts_of_tokens_that_come_thousands_of_times():
    d = make(2, 3, 1000, 30000, 0, 0, hot=True)
    check(d, apply(d))
    d = make(3, 3, 131072, 30000, 0, 0, generated=False, hot=True)
    check(d, apply(d))


def test_padding_tokens_duplicate_and_foreign_biases():
    d = make(4, 5, 2000, 50, 40, 0)
    rng = np.random.default_rng(0)
    d["tokens"][rng.integers(0, len(d["tokens"]), 30)] = rng.choice([-1, 2000, 2 ** 31 - 1, -2 ** 31], 30)
    d["bias_token"][rng.integers(0, len(d["bias_token"]), 10)] = rng.choice([-1, 2000, 2 ** 31 - 1, -2 ** 31], 10)
    n = len(d["bias_token"])
    d["bias_token"][:n // 2] = rng.choice(d["tokens"][:5].clip(0, 1999), n // 2)   # the same few tokens again and again
    check(d, apply(d))
    a, b = apply(d), apply(d)
    assert all(np.array_equal(x, y) for x, y in zip(a[:3], b[:3]))


def test_a_long_list_of_biases_with_two_of_a_token_far_apart():
    V = 50000
    d = make(12, 3, V, 30, 0, 0)
    rng = np.random.default_rng(1)
    tok = np.concatenate([rng.permutation(V), rng.permutation(V)[:300]]).astype(np.int32)
    d["bias_token"], d["bias_value"] = tok, rng.standard_normal(len(tok)).astype(np.float32)
    d["bias_start"] = np.array([0, 0, len(tok), len(tok)], np.int64)
    check(d, apply(d))


def test_start_positions_outside_their_lists_are_clamped():
    d = make(5, 4, 500, 20, 5, 0)
    d["row_start"] = np.array([-5, 3, 10, 2 ** 60, 2 ** 62], np.int64)
    d["generated_start"] = np.array([-9, 2 ** 50, 11, 0], np.int64)
    d["bias_start"] = np.array([-3, 2, 2, 2 ** 40, 2 ** 41], np.int64)
    check(d, apply(d))


def test_infinities_nan_and_ties():
    V = 40000
    d = make(6, 8, V, 0, 0, 2)
    l = d["logits"]
    d["mask_row"][:] = -1
    l[0] = NEG                                   # nothing above -inf
    l[1, 777] = l[1, 39999] = np.inf             # +inf twice: the lower token
    l[2, 5] = np.nan                             # a NaN among numbers
    l[3] = np.nan
    l[4] = 2.5                                   # all equal
    l[5] = -0.0
    l[5, 20000] = 0.0                            # equal to -0
    l[6] = np.finfo(np.float32).min              # the type's lowest value
    l[7, ::2] = np.nan                           # NaN in masked places only
    bits = np.zeros(((V + 31) // 32) * 32, bool)
    bits[1:V:2] = True
    d["mask"][0] = np.packbits(bits, bitorder="little").view(np.int32)
    d["mask_row"][7] = 0
    got = apply(d)
    check(d, got)
    assert list(got[1][:7]) == [-1, 777, int(np.nanargmax(l[2])), -1, 0, 0, 0]
    assert got[2][0] == NEG and got[2][1] == np.inf and np.isnan(got[2][2]) and np.isnan(got[2][3])
    assert abs(got[2][4] - (2.5 + np.log(V))) < 1e-5 and np.isfinite(got[2][7])
    assert got[3] == m.STATUS_NAN_LOGIT
    assert apply(d, ("out",))[3] == 0            # reported where token or lse is asked for


def test_bad_mask_index_leaves_nothing_and_is_reported():
    d = make(7, 5, 900, 0, 0, 2)
    d["mask_row"][:] = [0, -1, 2, -2, 2 ** 31 - 1]
    got = apply(d)
    check(d, got)
    assert list(got[1][2:]) == [-1, -1, -1] and got[3] == m.STATUS_BAD_MASK_INDEX
    del d["mask_row"]   # mask t for row t
    d["mask"] = np.ascontiguousarray(np.repeat(d["mask"][:1], 5, 0))
    check(d, apply(d))


@pytest.mark.parametrize("pad_in,pad_out,shift", [(0, 0, 0), (1, 0, 0), (4, 3, 0), (5, 5, 1), (0, 4, 4)])
def test_pitches_and_alignment(pad_in, pad_out, shift):
    T, V = 9, 3001
    d = make(8, T, V, 60, 8, 2)
    wide = torch.full((T, V + pad_in + shift), 9.0, device="cuda")
    l = wide[:, shift:shift + V]
    l.copy_(torch.from_numpy(d["logits"]))
    buf = torch.full((T, V + pad_out + shift), 5.0, device="cuda")
    out = buf[:, shift:shift + V]
    token, lse = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, device="cuda")
    m.moe_q4_logits_apply(rules(d), l, out=out, token=token, lse=lse)
    check(d, (out.cpu().numpy(), token.cpu().numpy(), lse.cpu().numpy()))
    assert bool((buf[:, :shift] == 5).all()) and bool((buf[:, shift + V:] == 5).all())


def test_a_long_buffer_past_32_bit_offsets():
    """Rows whose first element lies past 2^31 elements of the buffer."""
    T, V, ld = 3, 1000, (1 << 30) + 4096 + 4
    wide = torch.empty((T - 1) * ld + V, device="cuda")   # 8.6 GB
    l = wide.as_strided((T, V), (ld, 1))
    d = make(9, T, V, 30, 4, 2)
    l.copy_(torch.from_numpy(d["logits"]))
    got = apply(d, ("out", "token", "lse"), logits=l, in_place=True)
    check(d, got)


def test_captured_with_growing_histories():
    """A captured step: the histories, masks and logits change in place between replays."""
    T, V = 6, 9000
    d = make(10, T, V, 40, 6, 3)
    dev = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in d.items()}
    R = m.LogitRules(**{k: v for k, v in dev.items() if k != "logits"})
    out, token, lse = torch.empty(T, V, device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, device="cuda")
    m.moe_q4_logits_apply(R, dev["logits"], out=out, token=token, lse=lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_q4_logits_apply(R, dev["logits"], out=out, token=token, lse=lse)
    for seed in (11, 12):
        new = make(seed, T, V, 40, 6, 3)
        for k in ("logits", "mask", "mask_row", "repetition"):
            d[k] = new[k]
            dev[k].copy_(torch.from_numpy(new[k]))
        d["tokens"] = d["tokens"][::-1].copy()
        dev["tokens"].copy_(torch.from_numpy(d["tokens"]))
        g.replay()
        torch.cuda.synchronize()
        check(d, (out.cpu().numpy(), token.cpu().numpy(), lse.cpu().numpy()))


def test_no_rows_and_refusals_of_the_binding():
    l = torch.zeros(0, 50, device="cuda")
    assert m.moe_q4_logits_apply(m.LogitRules(), l)[0].shape == (0, 50)
    l = torch.zeros(3, 50, device="cuda")
    with pytest.raises(ValueError):
        m.moe_q4_logits_apply(m.LogitRules(mask=torch.zeros(1, 1, dtype=torch.int32, device="cuda")), l)
    with pytest.raises(ValueError):
        m.moe_q4_logits_apply(m.LogitRules(repetition=torch.ones(2, device="cuda")), l)
    with pytest.raises(ValueError):
        m.moe_q4_logits_apply(m.LogitRules(), l.double())
    with pytest.raises(ValueError):
        m.moe_q4_logits_apply(m.LogitRules(), l, out=torch.zeros(3, 51, device="cuda"))
    with pytest.raises(m.MoeQ4Error):   # shifted against itself by a row
        buf = torch.zeros(4, 50, device="cuda")
        m.moe_q4_logits_apply(m.LogitRules(), buf[:3], out=buf[1:])
    with pytest.raises(m.MoeQ4Error):   # a mask a row, but not as many as rows
        m.moe_q4_logits_apply(m.LogitRules(mask=torch.zeros(2, 2, dtype=torch.int32, device="cuda")), l)
