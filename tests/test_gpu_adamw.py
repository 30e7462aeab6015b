"""mp_grad_norm and mp_adamw_step against the formulas in 64 bits.

Tolerances, from the operations' roundings (e = 2^-24 each; the betas, lr and
the other arguments are taken as the fp32 values they are passed as):

* the coefficient k that unscales and clips has at most 6 roundings, so
  u = g k at most 7, and m = m b1 + u (1 - b1) is off by at most
  e (2 |m b1| + 9 |u c1|), v by e (2 v b2 + 17 u^2 c2) (first order; one more
  rounding is allowed for in each);
* the weight's second term is good to 2^-20 of itself by its specification,
  plus what m and v are off by; the first term has three roundings;
* a norm's sum of squares has at most 2 + 3 + n / (threads) + 8 + 8 roundings of
  positive terms; a thread adds at most n / 8 vectors: the bound used is
  e (24 + n_thread) with the thread's vector count;
* 8-bit codes: y = |m| 127^2 / M is off by 16129 (|dm| + |m| dM / M) / M + 3 e y;
  the code has to be the one the 64-bit y and the same random number give,
  unless they decide closer than that error.
"""

import numpy as np
import pytest
import torch

from gpu_util import assert_same_bits

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


def f32(x):
    return float(np.float32(x))


def mix32(x):
    x = np.asarray(x, dtype=np.uint64) & 0xFFFFFFFF
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x846CA68B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def uniforms(seed, ordinal, n):
    key = mix32((int(seed) + (ordinal + 1) * 0x9E3779B9) & 0xFFFFFFFF)
    h = mix32((key + np.arange(n, dtype=np.uint64)) & 0xFFFFFFFF)
    return (h & 0xFFFF).astype(np.float64) / 65536, (h >> 16).astype(np.float64) / 65536


class Tensor:
    """One tensor's state on the device, and its values in 64 bits."""

    def __init__(self, n, bits=32, grad=torch.bfloat16, copy="e4m3", decay=0.1, seed=0, grad_std=0.65, zero_state=False):
        rng = np.random.default_rng(seed * 7919 + n)
        self.n, self.bits, self.decay, self.copy_kind = n, bits, decay, copy
        blocks = (n + 255) // 256
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.master = dev(rng.standard_normal(n).astype(np.float32) * 0.02)
        self.grad = dev(rng.standard_normal(n).astype(np.float32) * grad_std).to(grad)
        self.sm = self.sv = None
        if bits == 32:
            m = rng.standard_normal(n).astype(np.float32) * 3e-6
            v = (rng.standard_normal(n).astype(np.float32) * 1e-5) ** 2
            self.m, self.v = dev(m * (not zero_state)), dev(v * (not zero_state))
        else:
            self.m = dev(rng.integers(-127, 128, n, dtype=np.int8) * np.int8(not zero_state))
            self.v = dev(rng.integers(0, 256, n, dtype=np.uint8) * np.uint8(not zero_state))
            self.sm = dev((rng.uniform(0.5, 2, blocks) * 1e-5 / 127 ** 2 * (not zero_state)).astype(np.float32))
            self.sv = dev((rng.uniform(0.5, 2, blocks) * 1e-10 / 255.0 ** 4 * (not zero_state)).astype(np.float32))
        self.copy = self.scale = self.amax = None
        if copy == "e4m3":
            self.copy = torch.full((n,), 0x55, dtype=torch.uint8, device="cuda")
            self.scale = torch.tensor([2048.0], device="cuda")
            self.amax = torch.tensor([0.0], device="cuda")
        elif copy == "bf16":
            self.copy = torch.full((n,), 3.0, dtype=torch.bfloat16, device="cuda")

    def add_to(self, plan):
        plan.add(self.grad, self.master, self.m, self.v, self.sm, self.sv, self.copy, self.scale, self.amax,
                 weight_decay=self.decay)

    def wide(self):
        """(g, w, m, v) in 64 bits."""
        g, w = self.grad.double().cpu().numpy(), self.master.double().cpu().numpy()
        m, v = self.m.double().cpu().numpy(), self.v.double().cpu().numpy()
        if self.bits == 8:
            of = np.arange(self.n) // 256
            m = m * np.abs(m) * self.sm.double().cpu().numpy()[of]
            v = v ** 4 * self.sv.double().cpu().numpy()[of]
        return g, w, m, v


class Step:
    def __init__(self, fp8mp, tensors, S=65536.0, growth=0, t=10, b1=0.9, b2=0.95, lr=3e-4, eps=1e-8, max_norm=0.0,
                 seed=12345, found=0, interval=2000):
        self.fp8mp, self.tensors = fp8mp, tensors
        self.b1, self.b2, self.lr, self.eps, self.max_norm, self.interval = b1, b2, lr, eps, max_norm, interval
        self.S = torch.tensor([S], device="cuda")
        self.growth = torch.tensor([growth], dtype=torch.int32, device="cuda")
        self.found = torch.tensor([found], dtype=torch.int32, device="cuda")
        self.pows = torch.tensor([b1 ** t, b2 ** t], device="cuda")
        self.seed = torch.tensor([seed], dtype=torch.int32, device="cuda")
        self.norm = torch.zeros(1, device="cuda")
        self.ws = torch.zeros(fp8mp.mp_adamw_workspace_bytes() // 4, dtype=torch.int32, device="cuda")
        self.plan = fp8mp.AdamWTensors()
        for x in tensors:
            x.add_to(self.plan)

    def measure(self):
        self.fp8mp.mp_grad_norm(self.plan, self.norm, self.found, self.ws)

    def run(self):
        self.fp8mp.mp_adamw_step(self.plan, self.S, self.growth, self.found, self.pows, self.ws, lr=self.lr,
                                 beta1=self.b1, beta2=self.b2, eps=self.eps, seed=self.seed,
                                 grad_norm=self.norm if self.max_norm else None, max_norm=self.max_norm,
                                 growth_interval=self.interval)
        assert self.fp8mp.fp8mp_check() == 0

    def check(self):
        """Runs one step and compares everything it writes with 64 bits."""
        before = [x.wide() for x in self.tensors]
        amax = [0.0 if x.amax is None else x.amax.item() for x in self.tensors]
        S, pows, seed = self.S.item(), self.pows.double().cpu().numpy(), self.seed.item() & 0xFFFFFFFF
        k = 1.0 / S
        if self.max_norm:
            k *= min(1.0, f32(self.max_norm) / (self.norm.double().item() * k + 1e-6))
        self.run()
        b1, b2, lr, eps = f32(self.b1), f32(self.b2), f32(self.lr), f32(self.eps)
        bc1, bc2 = 1 - pows[0] * b1, 1 - pows[1] * b2
        for t, (x, (g, w, m, v)) in enumerate(zip(self.tensors, before)):
            if x.n == 0:
                continue
            u = g * k
            dm = E * (3 * np.abs(m * b1) + 10 * np.abs(u * (1 - b1)))
            dv = E * (3 * v * b2 + 18 * u * u * (1 - b2))
            m = m * b1 + u * (1 - b1)
            v = v * b2 + u * u * (1 - b2)
            if x.bits == 8:  # the codes' decoding rounds too: c^2, c^4 and their products with the steps
                dm, dv = dm + 2 * E * np.abs(m), dv + 4 * E * v
            den = np.sqrt(v / bc2) + eps
            term = lr / bc1 * m / den
            dden = np.sqrt((v + dv) / bc2) - np.sqrt(np.maximum(v - dv, 0) / bc2)
            new = w * (1 - lr * f32(x.decay)) - term
            dw = E * (4 * np.abs(w) + 2 * np.abs(new)) + np.abs(term) * (2.0 ** -20 + dden / den) + lr / bc1 * dm / den
            got = x.master.double().cpu().numpy()
            assert (np.abs(got - new) <= dw).all(), ("master", t, np.abs(got - new).max())
            if x.bits == 32:
                assert (np.abs(x.m.double().cpu().numpy() - m) <= dm).all(), ("m", t)
                assert (np.abs(x.v.double().cpu().numpy() - v) <= dv).all(), ("v", t)
            else:
                rm, rv = uniforms(seed, t, x.n)
                self._codes(x.m, x.sm, np.abs(m), dm, rm, 2, 127, np.sign(m), ("m codes", t))
                self._codes(x.v, x.sv, v, dv, rv, 4, 255, np.ones(x.n), ("v codes", t))
            if x.amax is not None and x.n:
                assert x.amax.item() == max(amax[t], np.abs(got).max()), ("amax", t)
            self._copy(x, got, t)
        assert_same_bits(self.pows.cpu().numpy(), np.float32([np.float32(pows[0]) * np.float32(self.b1),
                                                              np.float32(pows[1]) * np.float32(self.b2)]), "powers")
        assert self.seed.item() & 0xFFFFFFFF == (seed + 1) & 0xFFFFFFFF
        assert self.ws[0].item() == 0

    @staticmethod
    def _codes(codes, step, a, da, r, p, top, sign, what):
        got = codes.double().cpu().numpy()
        n = got.size
        blocks = (n + 255) // 256
        pad = lambda z: np.pad(z, (0, blocks * 256 - n)).reshape(blocks, 256)  # noqa: E731
        M, dM = pad(a).max(1), pad(da).max(1)
        s = step.double().cpu().numpy()
        assert (np.abs(s - M / float(top) ** p) <= (dM + 3 * E * M) / float(top) ** p).all(), what
        of = np.arange(n) // 256
        levels = float(top) ** p
        with np.errstate(divide="ignore", invalid="ignore"):
            y = np.where(M[of] > 0, a * levels / M[of], 0.0)
            dy = np.where(M[of] > 0, levels * (da + a * dM[of] / M[of]) / M[of], 0.0) + 4 * E * y

        def code(y):
            c = np.floor(y ** (1.0 / p) + 1e-12)
            c = np.where((c + 1) ** p <= y, c + 1, np.where(c ** p > y, c - 1, c))
            c = np.minimum(c, top)
            c = np.where((c < top) & (r * ((c + 1) ** p - c ** p) < y - c ** p), c + 1, c)
            return np.maximum(c, 1) if p == 4 else c

        lo, hi = code(np.maximum(y - dy, 0)), code(y + dy)
        lo, hi = np.where(y > 0, lo, 0), np.where(y > 0, hi, 0)
        mag = np.abs(got)
        assert ((mag >= lo) & (mag <= hi)).all(), (what, int(((mag < lo) | (mag > hi)).sum()))
        assert (lo != hi).mean() < 0.02, what  # the comparison is sharp
        assert ((got == 0) | (np.sign(got) == sign) | (a <= da)).all(), what

    @staticmethod
    def _copy(x, w, t):
        if x.copy_kind == "bf16":
            want = torch.from_numpy(w.astype(np.float32)).to(torch.bfloat16)
            assert torch.equal(x.copy.cpu(), want), ("bf16 copy", t)
        elif x.copy_kind == "e4m3":
            want = (torch.from_numpy(w.astype(np.float32)) * x.scale.cpu()).clamp(-448, 448).to(torch.float8_e4m3fn)
            assert torch.equal(x.copy.cpu(), want.view(torch.uint8)), ("E4M3 copy", t)


SIZES = [1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 3839, 3840, 3841, 5000, 7680, 70001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("n", SIZES)
def test_one_tensor(cuda_lib, bits, n):
    x = Tensor(n, bits, seed=1)
    st = Step(cuda_lib, [x])
    for _ in range(3):
        st.check()


@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("copy", ["e4m3", "bf16", None])
def test_many_tensors_of_both_kinds(cuda_lib, grad, copy):
    tensors = [Tensor(n, bits, grad, copy, decay=0.1 * (i % 2), seed=i)
               for i, (n, bits) in enumerate((n, bits) for n in [0, *SIZES] for bits in (32, 8, 8))]
    st = Step(cuda_lib, tensors, max_norm=1e-3)
    st.measure()
    st.check()
    st.check()


@pytest.mark.parametrize("count", [31, 33, 281, 600, 1101])
def test_counts_that_need_several_launches(cuda_lib, count):
    tensors = [Tensor(1 + (37 * i) % 600, 8 if i % 3 == 0 else 32, seed=i) for i in range(count)]
    st = Step(cuda_lib, tensors, max_norm=1e-4)
    st.measure()
    total = sum(float((x.grad.double() ** 2).sum()) for x in tensors)
    assert abs(st.norm.item() - total ** 0.5) <= 40 * E * total ** 0.5
    st.check()
    assert st.growth.item() == 1


def codes_in_fp32(x, y, power, top, r):
    """The header's rounding in fp32 operations, each rounded once."""
    c = np.minimum(np.floor(y ** (1.0 / (2 if top == 127 else 4))), top).astype(np.float32)
    one = np.float32(1)
    c = np.where(power(c + one) <= y, c + one, c)
    c = np.minimum(np.where(power(c) > y, c - one, c), np.float32(top))
    lo = power(c)
    up = r.astype(np.float32) * (power(c + one) - lo) < y - lo
    return np.minimum(np.where(up, c + one, c), np.float32(top))


@pytest.mark.parametrize("clip", [0.0, 1e-3, 1e-5])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
def test_8_bit_moments_bit_for_bit(cuda_lib, grad, clip):
    """Moments, steps and codes equal those of the documented operations in
    fp32, every one rounded once (no product joins a sum unrounded). A small
    clip leaves gradients far below the moments: then all of a block decay
    alike, and nearly every code lies at the edge of its cell."""
    f = np.float32
    n = 256 * 1200
    x = Tensor(n, 8, grad, seed=31, copy=None)
    st = Step(cuda_lib, [x], max_norm=clip)
    st.measure()
    for _ in range(3):
        g, cm, cv = x.grad.float().cpu().numpy(), x.m.cpu().numpy().astype(f), x.v.cpu().numpy().astype(f)
        sm, sv = (np.repeat(s.cpu().numpy(), 256) for s in (x.sm, x.sv))
        pows, seed = st.pows.cpu().numpy(), st.seed.item() & 0xFFFFFFFF
        k = f(1) / f(st.S.item())
        if clip:
            c = f(clip) / (f(st.norm.item()) * k + f(1e-6))
            k = k * c if c < 1 else k
        b1, b2 = f(0.9), f(0.95)
        u = g * k
        m = (cm * np.abs(cm)) * sm * b1 + u * (f(1) - b1)
        v = ((cv * cv) * (cv * cv)) * sv * b2 + (u * u) * (f(1) - b2)
        st.run()
        M, V = np.abs(m).reshape(-1, 256).max(1), v.reshape(-1, 256).max(1)
        assert_same_bits(x.sm.cpu().numpy(), M / f(16129), "steps of m")
        assert_same_bits(x.sv.cpu().numpy(), V / f(4228250624.0), "steps of v")
        rm, rv = uniforms(seed, 0, n)
        im, iv = np.repeat(f(16129) / M, 256), np.repeat(f(4228250624.0) / V, 256)
        want = codes_in_fp32(x, np.abs(m) * im, lambda c: c * c, 127, rm)
        assert_same_bits(x.m.cpu().numpy(), np.where(m < 0, -want, want).astype(np.int8), "codes of m")
        want = codes_in_fp32(x, v * iv, lambda c: (c * c) * (c * c), 255, rv)
        assert_same_bits(x.v.cpu().numpy(), np.where(v > 0, np.maximum(want, 1), want).astype(np.uint8), "codes of v")
        assert np.array_equal(pows, np.float32(pows))


@pytest.mark.parametrize("seed", [31, 2 ** 31 - 1, -1])
def test_powers_and_seed_advance_with_every_step(cuda_lib, seed):
    """Bit for bit; a skipped step leaves them."""
    st = Step(cuda_lib, [Tensor(5000, 8, seed=1), Tensor(300, 32, seed=2)], max_norm=1e-3, seed=seed)
    st.measure()
    pows, want_seed = st.pows.cpu().numpy(), seed
    for found in (0, 0, 1, 0):
        st.found.fill_(found)
        st.run()
        if not found:
            pows = pows * np.float32([st.b1, st.b2])
            want_seed = (want_seed + 1 + 2 ** 31) % 2 ** 32 - 2 ** 31
        assert_same_bits(st.pows.cpu().numpy(), pows, "powers")
        assert st.seed.item() == want_seed


def test_no_tensors_at_all(cuda_lib):
    st = Step(cuda_lib, [], growth=4)
    st.norm.fill_(7.0)
    st.measure()
    assert st.norm.item() == 0.0 and st.found.item() == 0
    st.run()
    assert st.growth.item() == 5
    st.seed = None  # not needed without 8-bit moments
    st.run()
    assert st.growth.item() == 6


def test_scales_at_any_offset(cuda_lib):
    """The steps of the 8-bit moments need 4-byte alignment only."""
    x = Tensor(40000, 8, seed=21)
    for name in ("sm", "sv"):
        s = getattr(x, name)
        room = torch.zeros(s.numel() + 1, device="cuda")
        room[1:] = s
        setattr(x, name, room[1:])
    st = Step(cuda_lib, [x])
    st.check()
    st.check()


def test_large_tensors_of_both_kinds(cuda_lib):
    tensors = [Tensor(1500001, bits, grad, copy, seed=i) for i, (bits, grad, copy) in enumerate(
        [(8, torch.bfloat16, "e4m3"), (32, torch.float32, "bf16"), (8, torch.float32, "bf16"), (8, torch.bfloat16, None)])]
    st = Step(cuda_lib, tensors, max_norm=1e-3)
    st.measure()
    st.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_first_steps_from_zero_state(cuda_lib, bits):
    st = Step(cuda_lib, [Tensor(3001, bits, seed=3, zero_state=True)], t=0)
    for _ in range(3):
        st.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients_and_zero_state_only_decay(cuda_lib, bits):
    x = Tensor(700, bits, seed=5, zero_state=True, grad_std=0.0)
    w = x.master.clone()
    st = Step(cuda_lib, [x], t=0)
    st.check()
    assert (x.m == 0).all() and (x.v == 0).all()
    assert torch.allclose(x.master, w * (1 - 3e-4 * 0.1), rtol=1e-6, atol=0)


def test_blocks_too_small_for_a_scale_are_zero(cuda_lib):
    x = Tensor(512, 8, torch.float32, seed=6, zero_state=True, grad_std=0.0)
    x.grad[:256] = 1e-20  # u = 1.5e-25: v = 1e-51 leaves fp32, m = 1.5e-26 does not
    x.grad[256:] = 1e-9   # v = 1e-29 is below the smallest block
    st = Step(cuda_lib, [x], t=0)
    st.run()
    assert (x.v == 0).all() and (x.sv == 0).all()
    assert (x.m == 127).all() and (x.sm > 0).all()


def test_a_tiny_second_moment_keeps_a_code(cuda_lib):
    """v of one element is 1e-12 of its block's largest: its code stays 1, so
    that m / sqrt(v) of the next step stays bounded."""
    x = Tensor(256, 8, torch.float32, seed=7, zero_state=True, grad_std=0.0)
    x.grad[0], x.grad[1] = 1.0, 1e-6
    st = Step(cuda_lib, [x], t=0)
    st.run()
    assert x.v[0].item() == 255 and x.v[1].item() == 1 and (x.v[2:] == 0).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_overflow_skips_the_step(cuda_lib, bits):
    tensors = [Tensor(n, bits, seed=n) for n in (5, 4000)]
    tensors[1].grad[1234] = float("inf")
    st = Step(cuda_lib, tensors, S=1024.0, growth=9)
    st.measure()
    assert st.found.item() == 1
    keep = [[z.clone() for z in (x.master, x.m, x.v)] for x in tensors]
    pows, seed = st.pows.clone(), st.seed.clone()
    st.run()
    for x, old in zip(tensors, keep):
        for a, b in zip((x.master, x.m, x.v), old):
            assert torch.equal(a, b)
        # the copy is of the weights as they are, under a scale that may be new
        want = (x.master * x.scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(x.copy, want) and x.amax.item() == x.master.abs().max().item()
    assert st.S.item() == 512.0 and st.growth.item() == 0
    assert torch.equal(st.pows, pows) and torch.equal(st.seed, seed)
    tensors[1].grad[1234] = 0.25
    st.measure()
    assert st.found.item() == 0
    st.check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("copy", ["e4m3", "bf16", None])
def test_copies_of_a_skipped_step(cuda_lib, bits, copy):
    """More tensors than one launch takes, of odd sizes, some empty or without
    a copy; nothing past a copy's end is written."""
    sizes = [1, 7, 8, 2047, 2048, 2049, 0, 5000] * 40
    tensors = [Tensor(n, bits, copy=copy if i % 3 else None, seed=i) for i, n in enumerate(sizes)]
    spare = [x.copy for x in tensors]
    for x in tensors:
        if x.copy is not None:
            x.room = torch.cat([x.copy, x.copy.new_full((16,), 5)])
            x.copy = x.room[:x.n]
    del spare
    st = Step(cuda_lib, tensors, found=1)
    masters = [x.master.clone() for x in tensors]
    st.run()
    for x, w in zip(tensors, masters):
        assert torch.equal(x.master, w)
        if x.copy is None:
            continue
        if x.copy_kind == "bf16":
            want = w.to(torch.bfloat16)
        else:
            want = (w * x.scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
            assert x.n == 0 or x.amax.item() == w.abs().max().item()
        assert torch.equal(x.copy, want) and (x.room[x.n:] == 5).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
def test_nothing_past_the_ends(cuda_lib, bits, grad):
    """Every array between bytes that the step may not write, 16 bytes past a
    32-byte boundary: the results are those of arrays of their own."""
    sizes = [1, 7, 8, 9, 255, 256, 257, 2047, 2049, 5000, 40001]
    rooms = []

    def place(x):
        n = x.numel() * x.element_size()
        room = torch.full((n + 1024,), 0x5A, dtype=torch.uint8, device="cuda")
        at = 256 + (16 - (room.data_ptr() + 256)) % 32
        rooms.append((room, at, n))
        y = room[at:at + n].view(x.dtype)
        y.copy_(x)
        return y

    both = []
    for guarded in (False, True):
        tensors = [Tensor(n, bits, grad=grad, copy=("e4m3", "bf16")[i % 2], seed=i) for i, n in enumerate(sizes)]
        for x in tensors if guarded else []:
            for k in ("master", "grad", "m", "v", "sm", "sv", "copy"):
                if getattr(x, k) is not None:
                    setattr(x, k, place(getattr(x, k)))
        st = Step(cuda_lib, tensors, max_norm=1.0)
        st.measure()
        st.run()
        both.append((st, tensors))
    (st, plain), (guarded_st, guarded) = both
    assert torch.equal(st.norm, guarded_st.norm)
    for x, y in zip(plain, guarded):
        for k in ("master", "m", "v", "sm", "sv", "copy"):
            if getattr(x, k) is not None:
                assert torch.equal(getattr(x, k).view(torch.uint8), getattr(y, k).view(torch.uint8)), (x.n, k)
    for room, at, n in rooms:
        assert (room[:at] == 0x5A).all() and (room[at + n:] == 0x5A).all()


def test_loss_scale_grows(cuda_lib):
    st = Step(cuda_lib, [Tensor(100)], S=8.0, growth=1, interval=3)
    st.check()
    assert st.S.item() == 8.0 and st.growth.item() == 2
    st.check()
    assert st.S.item() == 16.0 and st.growth.item() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 8191, 8192, 8193, 3000017])
def test_norm(cuda_lib, dtype, n):
    st = Step(cuda_lib, [Tensor(n, grad=dtype, seed=2)])
    x = st.tensors[0]
    want = float((x.grad.double() ** 2).sum()) ** 0.5
    per_thread = (n // 8192 + 1) * 32 // (152 * 8) + 33
    got = []
    for _ in range(2):
        st.measure()
        got.append(st.norm.item())
    assert got[0] == got[1]  # fixed order
    assert abs(got[0] - want) <= E * (24 + per_thread) * want
    assert st.found.item() == 0 and (st.ws[:4] == 0).all()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan"), 3e38])
def test_norm_finds_overflow(cuda_lib, bad):
    st = Step(cuda_lib, [Tensor(20000, seed=i) for i in range(3)])
    st.tensors[2].grad[19999] = bad
    st.measure()
    assert st.found.item() == 1 and not np.isfinite(st.norm.item())
    st.tensors[2].grad[19999] = 1.0
    st.measure()
    assert st.found.item() == 0 and np.isfinite(st.norm.item())


def test_norm_past_2_64(cuda_lib):
    """64 gradients in one block of threads or in 64 blocks: a norm of 2^63, and one
    of 2^64, which counts as infinite either way."""
    n = 8192 * 64
    for scattered in (False, True):
        x = Tensor(n, grad=torch.float32, copy=None, grad_std=0.0)
        st = Step(cuda_lib, [x])
        places = torch.arange(64, device="cuda") * (8192 if scattered else 1)
        x.grad[places] = 2.0 ** 60  # the norm is 2^63
        st.measure()
        assert st.norm.item() == 2.0 ** 63 and st.found.item() == 0
        x.grad[places] = 2.0 ** 61  # 2^64
        st.measure()
        assert st.norm.item() == float("inf") and st.found.item() == 1, scattered


def test_rounding_is_unbiased(cuda_lib):
    """Over 400 seeds the stored moments' mean is the moment: the deviation of a
    mean of 400 two-valued codes is at most half a step / 20; 5 of those."""
    n, rounds = 2560, 400
    x = Tensor(n, 8, seed=11, copy=None)
    st = Step(cuda_lib, [x])
    state = [z.clone() for z in (x.master, x.m, x.v, x.sm, x.sv)]
    g, w, m, v = x.wide()
    k = 1.0 / 65536
    b1, b2 = f32(0.9), f32(0.95)
    m, v = m * b1 + g * k * (1 - b1), v * b2 + (g * k) ** 2 * (1 - b2)
    sums = np.zeros((2, n))
    for seed in range(rounds):
        for z, old in zip((x.master, x.m, x.v, x.sm, x.sv), state):
            z.copy_(old)
        st.seed.fill_(seed * 2654435761 % 2 ** 31)
        st.run()
        _, _, mq, vq = x.wide()
        sums += [mq, vq]
    of = np.arange(n) // 256
    sm, sv = x.sm.double().cpu().numpy()[of], x.sv.double().cpu().numpy()[of]
    cm, cv = np.sqrt(np.abs(m) / sm), (v / sv) ** 0.25
    step_m, step_v = (2 * cm + 1) * sm, ((cv + 1) ** 4 - cv ** 4) * sv
    assert (np.abs(sums[0] / rounds - m) <= 5 * step_m / 40 + 1e-6 * np.abs(m)).all()
    big = cv >= 1  # below, the code 1 is the smallest
    assert (np.abs(sums[1] / rounds - v) <= 5 * step_v / 40 + 1e-6 * v)[big].all()


def test_8_bit_moments_train_as_32_bit_ones_do(cuda_lib):
    """Least squares from the same start: the losses end alike."""
    torch.manual_seed(0)
    d = 512
    A = torch.randn(2048, d, device="cuda")
    target = torch.randn(d, device="cuda")
    losses = {}
    for bits in (32, 8):
        x = Tensor(d, bits, torch.float32, None, decay=0.0, seed=1, zero_state=True)
        x.master.zero_()
        st = Step(cuda_lib, [x], S=1.0, t=0, lr=1e-2, b2=0.95)
        for i in range(300):
            err = A @ (x.master - target)
            x.grad.copy_(A.T @ err / 2048)
            st.run()
        losses[bits] = float(((A @ (x.master - target)) ** 2).mean())
    start = float(((A @ target) ** 2).mean())
    assert losses[32] < 0.01 * start and losses[8] < 0.01 * start, (losses, start)


@pytest.mark.slow
def test_more_than_2_32_elements(cuda_lib):
    """One tensor of 2^32 + 10007 elements with 8-bit moments, zero but for the
    last 3000 elements: they and the random numbers of their places are right."""
    n, tail = 2 ** 32 + 10007, 3000
    z = lambda dtype: torch.zeros(n, dtype=dtype, device="cuda")  # noqa: E731
    blocks = (n + 255) // 256
    x = Tensor(1, 8, copy=None)
    x.n, x.grad, x.master, x.m, x.v = n, z(torch.bfloat16), z(torch.float32), z(torch.int8), z(torch.uint8)
    x.sm, x.sv = torch.zeros(blocks, device="cuda"), torch.zeros(blocks, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x.grad[-tail:] = torch.randn(tail, generator=g, device="cuda").to(torch.bfloat16)
    st = Step(cuda_lib, [x], t=0)
    st.measure()
    want = float(x.grad[-tail:].double().square().sum()) ** 0.5
    assert abs(st.norm.item() - want) <= 1e-6 * want and st.found.item() == 0
    seed = st.seed.item() & 0xFFFFFFFF
    st.run()
    assert not x.m[:-tail].any() and not x.v[:-tail].any() and not x.master[:-tail].any()
    u = x.grad[-tail:].double().cpu().numpy() / 65536.0
    m, v = (1 - f32(0.9)) * u, (1 - f32(0.95)) * u * u
    first = (n - tail) // 256  # its block's first elements are zero
    of = (np.arange(n - tail, n) // 256) - first
    M, V = (np.array([z[of == b].max() for b in range(of[-1] + 1)]) for z in (np.abs(m), v))
    key = mix32((seed + 0x9E3779B9) & 0xFFFFFFFF)
    i = np.arange(n - tail, n, dtype=np.uint64)
    h = mix32((key + (i & 0xFFFFFFFF) + (i >> 32) * 0x85EBCA77) & 0xFFFFFFFF)
    for got, y, p, top, r in ((x.m, np.abs(m) * 127.0 ** 2 / M[of], 2, 127, (h & 0xFFFF) / 65536.0),
                              (x.v, v * 255.0 ** 4 / V[of], 4, 255, (h >> 16) / 65536.0)):
        def code(y):
            c = np.minimum(np.floor(y ** (1.0 / p) + 1e-12), top)
            c = np.where(c ** p > y, c - 1, c)
            return np.where((c < top) & (r * ((c + 1) ** p - c ** p) < y - c ** p), c + 1, c)

        lo, hi = code(y * (1 - 2.0 ** -20)), code(y * (1 + 2.0 ** -20))
        if p == 4:
            lo, hi = np.maximum(lo, 1), np.maximum(hi, 1)
        mag = np.abs(got[-tail:].double().cpu().numpy())
        assert ((mag >= lo) & (mag <= hi)).all()


def test_another_stream(cuda_lib):
    tensors = [Tensor(5000, 8, seed=1), Tensor(5000, 32, seed=2)]
    st = Step(cuda_lib, tensors, max_norm=1e-3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        st.measure()
        st.check()
    torch.cuda.current_stream().wait_stream(side)


def test_graph_replay_is_the_call(cuda_lib):
    a = Step(cuda_lib, [Tensor(3000, 8, seed=4), Tensor(900, 32, seed=5)], max_norm=1e-3)
    b = Step(cuda_lib, [Tensor(3000, 8, seed=4), Tensor(900, 32, seed=5)], max_norm=1e-3)

    def both(st):
        st.measure()
        st.fp8mp.mp_adamw_step(st.plan, st.S, st.growth, st.found, st.pows, st.ws, lr=st.lr, beta1=st.b1, beta2=st.b2,
                               eps=st.eps, seed=st.seed, grad_norm=st.norm, max_norm=st.max_norm)

    for _ in range(3):
        both(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(b)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(a.tensors, b.tensors):
        for p, q in zip((x.master, x.m, x.v, x.copy), (y.master, y.m, y.v, y.copy)):
            assert torch.equal(p, q)
    assert torch.equal(a.seed, b.seed) and torch.equal(a.pows, b.pows)


def test_new_gradients(cuda_lib):
    tensors = [Tensor(100, seed=1), Tensor(300, 8, seed=2)]
    st = Step(cuda_lib, tensors)
    for x in tensors:
        x.grad = torch.randn(x.n, device="cuda")  # fp32 now
    st.plan.set_grads([x.grad for x in tensors])
    st.check()
