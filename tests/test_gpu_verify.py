"""Verification of drafted blocks against the fp64 statement.

Whole numbers must be equal.  A block whose result hangs on less than the fp32 rounding of p and q
(relative 2^-23 * (64 + |z|max) for the softmax's exponent, sum and quotient) is excused; prob is
held to four times that."""
import numpy as np
import pytest
import torch

from jacobi_speculative_decode_gb300 import xp
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu


def make_head(V, B, N, dtype):
    r, dt = 8, xp.torch_dtype(dtype)
    shapes = dict(w1=(V, r), down_h=(r, r), down_g=(r, r), in_proj=(r, 3 * r), mix_L=(r, B, B),
                  w_gate=(r, r), w_up=(r, r), w_down=(r, r), w2=(V, r))
    w = {k: torch.zeros(s, dtype=dt, device="cuda") for k, s in shapes.items()}
    return xp.Head(dict(V=V, hidden=r, r=r, H=r, B=B), w, dtype, N)


class Case:
    def __init__(self, N, B, V, dtype="bf16", drafts=True, seed=0, n_draft=None, greedy=(), pad=0,
                 spread=2.5):
        g = np.random.default_rng(seed)
        self.N, self.B, self.V, self.dtype = N, B, V, dtype
        dt = xp.torch_dtype(dtype)
        wide = torch.from_numpy(g.normal(size=(N, B, V + pad)).astype(np.float32) * spread).to(dt)
        self.target = wide.cuda()[:, :, pad:]
        heat = g.uniform(0.6, 1.5, N).astype(np.float32)
        heat[list(greedy)] = 0
        self.temperature = heat
        self.draft = None
        self.blk = g.integers(0, V, (N, B))
        if drafts:
            near = wide[:, :-1, pad:].float().numpy() + g.normal(size=(N, B - 1, V)) * 0.5
            self.draft = near.reshape(N * (B - 1), V).astype(np.float32)
            hot = np.where(heat > 0, heat, 1)[:, None, None]
            race = near / hot - np.log(g.exponential(size=near.shape)) * (heat > 0)[:, None, None]
            self.blk[:, 1:] = race.argmax(-1)
        else:   # drafts the target likes
            self.blk[:, 1:] = wide[:, :-1, pad:].float().numpy().argmax(-1)
        self.u = g.random((N, B - 1)).astype(np.float32)
        self.noise = np.maximum(g.exponential(size=(N, V)), 1e-20).astype(np.float32)
        self.n_draft = None if n_draft is None else np.asarray(n_draft, np.int32)

    def run(self, head=None, ws=None, stream=None):
        N, B = self.N, self.B
        cu = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        head = head or make_head(self.V, B, N, self.dtype)
        ws = head.verify_workspace(N) if ws is None else ws
        tokens = torch.full((N, B), 77, dtype=torch.int64, device="cuda")
        counts = torch.full((N,), 77, dtype=torch.int32, device="cuda")
        prob = torch.full((N, B - 1), 77.0, device="cuda")
        xp.xp_verify_drafts(head.handle, self.target, cu(self.draft), cu(self.blk), cu(self.n_draft),
                            cu(self.temperature), cu(self.u), cu(self.noise), tokens, counts, prob,
                            ws, stream)
        self.error = xp.xp_get_error(head.handle, stream)
        return tokens.cpu().numpy(), counts.cpu().numpy(), prob.cpu().numpy()

    def want(self):
        return S.verify(self.target.float().cpu().numpy(), self.draft, self.blk, self.n_draft,
                        self.temperature, self.u, self.noise)

    def check(self, got=None):
        tokens, counts, prob = got or self.run()
        wt, wc, wp, margin = self.want()
        z = self.target.float()
        z = z[z.abs() < 1e4]               # larger ones are masks: their weights are 0 or 1 exactly
        top = float(z.abs().max()) if z.numel() else 0.0
        eps = 2.0 ** -23 * (64 + 2 * top / 0.6)
        sure = margin > 4 * eps
        assert sure.sum() >= self.N - 1 - self.N // 50
        assert np.array_equal(tokens[sure], wt[sure]) and np.array_equal(counts[sure], wc[sure])
        assert np.all(np.abs(prob - wp)[sure] <= 4 * eps * wp[sure])


CASES = [
    dict(N=1, B=2, V=1), dict(N=1, B=2, V=2, drafts=False), dict(N=3, B=2, V=7),
    dict(N=5, B=8, V=500, greedy=(0, 3)), dict(N=5, B=8, V=500, drafts=False, greedy=(1,)),
    dict(N=9, B=4, V=8192), dict(N=9, B=4, V=8193, drafts=False), dict(N=4, B=16, V=20001, greedy=(2,)),
    dict(N=70, B=5, V=3001, drafts=False), dict(N=6, B=5, V=4104, pad=3),
    dict(N=6, B=5, V=4100, n_draft=[0, 1, 2, 3, 4, 4]), dict(N=2, B=64, V=1000, spread=0.5),
    dict(N=300, B=3, V=900),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", CASES, ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
def test_matches_the_statement(kw, dtype):
    c = Case(dtype=dtype, seed=len(str(kw)), **kw)
    c.check()
    assert c.error == xp.XP_OK


def test_full_vocabulary():
    Case(N=3, B=16, V=151936, seed=4, greedy=(1,)).check()


def test_masked_and_odd_logits():
    # masks of -inf and of the type's lowest value, NaN, +inf, and a row with one token left
    c = Case(N=8, B=4, V=700, seed=5, dtype="f32")
    t = c.target
    t[0, :, 5:] = -np.inf
    t[1, :, ::2] = torch.finfo(torch.float32).min
    t[2, :, 100:200] = np.nan
    t[3, 0, 9] = np.inf
    t[4, :, 1:] = -np.inf
    t[5, :, 699] = -0.0
    c.draft[5 * 3:6 * 3, 10:] = -np.inf
    c.temperature[6] = 0
    t[6, :, 3] = t[6, :, 650] = 1e30
    c.blk[0:5, 1:] = c.blk[0:5, 1:] % 5
    c.check()
    assert c.error == xp.XP_OK


def test_row_that_leaves_no_token():
    c = Case(N=3, B=3, V=50, seed=6)
    c.target[0, 0] = -np.inf
    c.target[1] = np.nan
    c.temperature[1] = 0
    tokens, counts, _ = c.run()
    assert tokens[:2].tolist() == [[-1] * 3] * 2 and counts[:2].tolist() == [0, 0]
    assert c.error == xp.XP_EEMPTY
    assert np.array_equal(tokens[2], c.want()[0][2])


def test_bad_drafted_ids_are_rejected():
    c = Case(N=4, B=4, V=60, seed=7, drafts=False)
    c.blk[0, 1], c.blk[1, 2], c.blk[2, 1] = -1, 60, 1 << 40
    c.check()
    assert c.error == xp.XP_EBADTOKEN


def test_draft_counts_are_clamped():
    c = Case(N=4, B=4, V=60, seed=8, n_draft=[-3, 9, 3, 0])
    c.check()
    assert c.error == xp.XP_ELENGTH


def test_certain_and_impossible_drafts():
    # p == q accepts everything (u < 1); a draft that p excludes is never accepted, u = 0 included
    c = Case(N=4, B=6, V=333, seed=9, dtype="f32")
    c.draft = c.target[:, :-1].cpu().numpy().reshape(-1, c.V).copy()
    c.u[:] = np.float32(1 - 2 ** -20)
    c.u[1] = 0
    x = c.blk[1, 1]
    c.target[1, 0, x] = -np.inf
    tokens, counts, _ = c.run()
    assert counts.tolist() == [6, 1, 6, 6] and tokens[1, 0] != x


def test_workspace_is_left_ready_and_shared_by_batches():
    head = make_head(600, 6, 40, "bf16")
    ws = head.verify_workspace(40)
    for seed, N in ((1, 40), (2, 7), (3, 40)):
        c = Case(N=N, B=6, V=600, seed=seed, drafts=seed != 2)
        first = c.run(head, ws)
        again = c.run(head, ws)
        assert all(np.array_equal(a, b) for a, b in zip(first, again))
        c.check(first)


def test_other_stream_and_graph():
    c = Case(N=5, B=5, V=900, seed=12)
    head = make_head(900, 5, 5, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.check(c.run(head))
    cu = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    args = [c.target, cu(c.draft), cu(c.blk), None, cu(c.temperature), cu(c.u), cu(c.noise)]
    out = [torch.zeros(5, 5, dtype=torch.int64, device="cuda"),
           torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(5, 4, device="cuda")]
    ws = head.verify_workspace(5)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        xp.xp_verify_drafts(head.handle, *args, *out, ws)
    for _ in range(2):
        out[0].zero_()
        g.replay()
        c.check(tuple(t.cpu().numpy() for t in out))


def test_refusals():
    c = Case(N=2, B=4, V=64, seed=1)
    head = make_head(64, 4, 2, "bf16")
    cu = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    ws = head.verify_workspace(2)
    out = [torch.zeros(2, 4, dtype=torch.int64, device="cuda"),
           torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, 3, device="cuda")]
    ok = dict(target=c.target, draft=cu(c.draft), blk=cu(c.blk), n_draft=None, temperature=None,
              u=cu(c.u), noise=cu(c.noise), tokens=out[0], counts=out[1], prob=out[2], ws=ws)

    def code(**kw):
        try:
            xp.xp_verify_drafts(head.handle, **{**ok, **kw})
        except xp.XPError as e:
            return e.code
        return xp.XP_OK

    assert code() == xp.XP_OK
    assert code(ws=ws[:ws.numel() - 256]) == xp.XP_ECAPACITY
    assert code(ws=ws[8:]) == xp.XP_EINVAL
    assert code(target=c.target.float()) == xp.XP_EINVAL               # not the head's type
    assert code(target=c.target[:, :3], tokens=out[0]) == xp.XP_EINVAL   # another block size
    assert code(target=c.target.repeat(2, 1, 1), draft=None, blk=cu(c.blk).repeat(2, 1),
                u=cu(c.u).repeat(2, 1), noise=cu(c.noise).repeat(2, 1), tokens=out[0].repeat(2, 1),
                counts=out[1].repeat(2), prob=None) == xp.XP_ECAPACITY   # above max_N
    for bad in (dict(u=cu(c.u).double()), dict(blk=cu(c.blk).int()), dict(noise=cu(c.noise)[:, :60]),
                dict(tokens=out[0][:1]), dict(draft=cu(c.draft)[:, :60])):
        with pytest.raises(ValueError):
            code(**bad)
