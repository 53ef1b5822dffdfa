"""The end of a decode step as a server runs it: the W4A8 LM head, each row's
low-rank adapter added in place, each row's logit rules, the greedy token and
its log-probability; then the same as one captured graph over several steps
in which the histories grow; and an adapter beside the expert layer."""
import numpy as np
import pytest
import torch

import oracle
import synth

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import quantized_moe_q4_b200 as m  # noqa: E402

T, H, V, R, NA, LONG = 8, 512, 4001, 16, 3, 64


class Step:
    """Buffers and calls of one decode step; row t's history is tokens[t * LONG : row_end]."""

    def __init__(self):
        rng = np.random.default_rng(3)
        self.W = synth._q4_0_matrix(np.random.Generator(np.random.PCG64(5)), V, H // 32)
        self.a = (rng.standard_normal((NA, R, H)) / np.sqrt(H)).astype(np.float16)
        self.b = (rng.standard_normal((NA, V, R)) * 0.5).astype(np.float16)
        self.scale = np.array([1.0, 0.5, 2.0], np.float32)
        self.ids = np.array([0, 2, -1, 1, 1, -1, 0, 2], np.int32)
        self.Wd = torch.from_numpy(self.W).cuda()
        self.A = m.Adapters(torch.from_numpy(self.a).cuda(), torch.from_numpy(self.b).cuda(), torch.from_numpy(self.scale).cuda())
        self.idsd = torch.from_numpy(self.ids).cuda()
        self.x = torch.zeros(T, H, device="cuda")
        # histories in fixed slots, padded with -1 behind the last token
        self.tokens = torch.full((T * LONG,), -1, dtype=torch.int32, device="cuda")
        self.start = torch.arange(T + 1, device="cuda") * LONG
        self.rep = torch.linspace(1, 1.7, T, device="cuda")
        self.pres = torch.linspace(0, 1, T, device="cuda")
        self.freq = torch.linspace(0.5, 0, T, device="cuda")
        self.mask = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, (2, (V + 31) // 32)).astype(np.int32)).cuda()
        self.mask_row = torch.tensor([-1, 0, 1, -1, 0, 1, -1, -1], dtype=torch.int32, device="cuda")
        self.rules = m.LogitRules(tokens=self.tokens, row_start=self.start, repetition=self.rep, presence=self.pres,
                                  frequency=self.freq, mask=self.mask, mask_row=self.mask_row)
        self.logits = torch.empty(T, V, device="cuda")
        self.token = torch.empty(T, dtype=torch.int32, device="cuda")
        self.lse = torch.empty(T, device="cuda")
        self.ws = m.alloc_workspace(m.moe_q4_gemv_workspace_bytes(T, H))
        self.aws = m.alloc_workspace(m.moe_q4_adapters_workspace_bytes(self.A, T))

    def run(self):
        m.moe_q4_gemv(self.Wd, self.x, y=self.logits, workspace=self.ws)
        m.moe_q4_adapters_apply(self.A, self.x, self.idsd, base=self.logits, y=self.logits, workspace=self.aws)
        m.moe_q4_logits_apply(self.rules, self.logits, out=self.logits, token=self.token, lse=self.lse)

    def expected(self):
        """(processed logits in binary64, scale of the rounding errors) for the buffers as they are."""
        x = self.x.cpu().numpy()
        q, d, _ = oracle.quantize_q8_0(x)
        l = np.stack([oracle.q4_matvec(self.W, q[t], d[t]) for t in range(T)]).astype(np.float64)
        big = np.sqrt(np.mean(l ** 2))
        for t in range(T):
            if self.ids[t] >= 0:
                e = self.ids[t]
                l[t] += self.scale[e] * (self.b[e].astype(np.float64) @ (self.a[e].astype(np.float64) @ x[t].astype(np.float64)))
            h = self.tokens[t * LONG:(t + 1) * LONG].cpu().numpy()
            c = np.bincount(h[h >= 0], minlength=V)
            rep, pres, freq = (float(v[t]) for v in (self.rep, self.pres, self.freq))
            l[t] = np.where(c > 0, np.where(l[t] > 0, l[t] / rep, l[t] * rep) - freq * c - pres, l[t])
            r = int(self.mask_row[t])
            if r >= 0:
                bits = np.unpackbits(self.mask[r].cpu().numpy().view(np.uint8), bitorder="little")[:V]
                l[t][bits == 0] = -np.inf
        return l, big

    def check(self):
        l, big = self.expected()
        got = self.logits.cpu().numpy()
        assert np.array_equal(np.isinf(got), np.isinf(l))
        fine = np.isfinite(l)
        # the LM head is within 1e-5 of the row scale of the oracle; the rest adds roundings of 2^-24 each
        assert np.all(np.abs(got[fine] - l[fine]) <= 2e-5 * (np.abs(l[fine]) + big))
        tok, lse = self.token.cpu().numpy(), self.lse.cpu().numpy()
        assert np.array_equal(tok, got.argmax(1))   # of the logits that the call left
        for t in range(T):
            top = l[t].max()
            assert l[t, tok[t]] >= top - 4e-5 * (abs(top) + big)
            assert abs(lse[t] - (top + np.log(np.exp(l[t] - top).sum()))) <= 4e-5 * (abs(top) + big)
        return tok


def test_a_step_and_then_captured_steps_with_growing_histories():
    s = Step()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    s.x.copy_(torch.randn(T, H, device="cuda", generator=g))
    s.run()
    torch.cuda.synchronize()
    s.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    place = torch.arange(T, device="cuda") * LONG
    for step in range(6):
        graph.replay()
        torch.cuda.synchronize()
        s.check()
        # the chosen tokens join the histories; the same hidden state again, so that the penalties must show
        s.tokens[place + step] = s.token
        if step == 3:
            s.x.copy_(torch.randn(T, H, device="cuda", generator=g))
    hist = s.tokens.cpu().numpy().reshape(T, LONG)
    assert len(set(hist[7, :3])) > 1   # a penalty of 1.7 and 1 moves row 7 on from its first choice
    assert int(s.aws[:4].view(torch.int32)) == 0


@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_an_adapter_beside_the_expert_layer(tokens):
    """y = layer(x) + adapter(x) in place on the layer's output."""
    x, lw = synth.random_layer(seed=9, H=512, F=256, E=16, k=4, shared=True, T=tokens)
    L = m.Layer.from_host(lw)
    xd = torch.from_numpy(x).cuda()
    y = m.moe_q4_ffn_forward(L, xd)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    a = (torch.randn(4, 8, 512, device="cuda", generator=g) / 512 ** 0.5).bfloat16()
    b = (torch.randn(4, 512, 8, device="cuda", generator=g)).bfloat16()
    ids = torch.randint(-1, 4, (tokens,), device="cuda", generator=g).int()
    plain = y.double()
    e = ids.clamp(min=0).long()
    u = torch.einsum("trh,th->tr", a[e].double(), xd.double())
    d = torch.einsum("tnr,tr->tn", b[e].double(), u) * (ids >= 0)[:, None]
    size = plain.abs() + torch.einsum("tnr,tr->tn", b[e].double().abs(), torch.einsum("trh,th->tr", a[e].double().abs(), xd.double().abs()))
    m.moe_q4_adapters_apply(m.Adapters(a, b), xd, ids, base=y, y=y)
    assert bool(((y.double() - plain - d).abs() <= (512 / 16 + 2 * 8 + 64) * 2.0 ** -24 * size).all())
