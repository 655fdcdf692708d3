"""The 8-bit pool without a GPU: the oracle's format against closed forms and
torch's e4m3, where the decode kernel finds what the copies land, the refusals of
the C calls and of the binding."""

import ctypes

import numpy as np
import pytest

import oracle
from paged_kv_cache_hkv_gb300 import binding, build
from quant_cases import odd_rows
from test_abi_host import FAKE, MISALIGNED, _layout
from test_abi_host import header_define as E

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return binding.load()


# ------------------------------------------------------------------ the format
def test_codes_are_torchs_e4m3():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.e4m3_values(codes), want, equal_nan=True)


def test_rounding_is_torchs_and_the_scale_the_least_that_reaches():
    bits = odd_rows(400, 3, 64, 1)
    codes, scales = oracle.quantise_rows(bits)
    x = oracle.bf16_bits_to_f64(bits)
    fine = np.isfinite(x).all(-1)
    e = scales.astype(int) - 127
    assert (scales[~fine] == 255).all() and not codes[~fine].any()
    top = np.abs(x[fine]).max(-1)
    assert (top <= 448 * 2.0 ** e[fine]).all() and (e[fine] >= -117).all()
    assert ((e[fine] == -117) | (top > 224 * 2.0 ** e[fine])).all()
    y = torch.from_numpy(x[fine] / 2.0 ** e[fine][:, None]).float().to(torch.float8_e4m3fn)
    assert np.array_equal(y.view(torch.uint8).numpy(), codes[fine])


def test_values_are_bf16_and_survive_a_second_write():
    codes, scales = oracle.quantise_rows(odd_rows(300, 2, 128, 2))
    bits = oracle.quant_pool_bits(codes, scales)
    again = oracle.quantise_rows(bits)
    assert np.array_equal(oracle.quant_values(*again), oracle.quant_values(codes, scales),
                          equal_nan=True)


def test_the_error_is_half_a_step():
    bits = odd_rows(300, 2, 64, 3)
    codes, scales = oracle.quantise_rows(bits)
    x, y = oracle.bf16_bits_to_f64(bits), oracle.quant_values(codes, scales)
    fine = (scales != 255)
    unit = 2.0 ** (scales[fine].astype(float) - 127)[:, None]
    assert (np.abs(x[fine] - y[fine]) <= np.maximum(2.0 ** -4 * np.abs(x[fine]), 2.0 ** -10 * unit)).all()


def test_write_skips_padding_and_read_leaves_it():
    codes, scales = oracle.quantise_rows(odd_rows(8 * 2 * 16, 2, 64, 4).reshape(8, 2, 16, 2, 64))
    k = odd_rows(3, 2, 64, 5)
    after = oracle.quant_write(codes, scales, k, k, [5, -1, 127])
    changed = np.argwhere((after[0] != codes).any(axis=(3, 4)) | (after[1] != scales).any(axis=3))
    assert {(int(b), int(o)) for b, _, o in changed} <= {(0, 5), (7, 15)}
    out = oracle.quant_read(k, k.copy(), *after, [-4, 5, 127])
    assert np.array_equal(out[0][0], k[0])
    assert np.array_equal(out[0][1], oracle.quant_pool_bits(*(x[0, 0, 5] for x in after)))


# ------------------------------------------------------------------ where the copies land
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("KH", [1, 3, 8])
def test_ldmatrix_finds_each_key_and_dim_without_bank_conflicts(D, B, KH):
    """The decode kernel's addresses restated: a copy of a box {D, 16 rows (8 for
    8-token blocks), KH heads, K and V} lands innermost first and swizzled (16-byte
    units of a 128 or 64 byte row XORed with address bits 7.. ); lane l of an
    ldmatrix reads 16 bytes at k_off ^ (kk << 5)."""
    rows = 8 if B == 8 else 16
    stage = {}  # byte address -> (K|V, head, key, dim)
    for copy in range(2 if B == 8 else 1):
        base = copy * 16 * KH * D
        for kv in range(2):
            for h in range(KH):
                for r in range(rows):
                    for d in range(D):
                        a = base + ((kv * KH + h) * rows + r) * D + d
                        a ^= ((a >> 7) & (7 if D == 128 else 3)) << 4
                        assert a not in stage
                        stage[a] = (kv, h, copy * 8 + r, d)
    assert len(stage) == 32 * KH * D
    group = 16 * KH * D if B == 8 else 8 * D
    step = (8 if B == 8 else 16) * KH * D
    for h in range(KH):
        for kk in range(D // 32):
            for kv in range(2):
                lanes = []
                for lane in range(32):
                    row8 = lane & 7
                    swz = row8 if D == 128 else row8 >> 1
                    off = (8 if B == 8 else 16) * h * D + row8 * D + (group if (lane >> 3) & 1 else 0)
                    off += ((lane >> 4) ^ swz) << 4
                    a = (off + kv * step) ^ (kk << 5)
                    key = row8 + 8 * ((lane >> 3) & 1)
                    dim = 16 * (2 * kk + (lane >> 4))
                    assert [stage[a + i] for i in range(16)] == [(kv, h, key, dim + i) for i in range(16)]
                    lanes.append(a)
                for q in range(4):  # eight lanes a phase: 128 bytes in 32 different banks
                    assert len({(a // 16) % 8 for a in lanes[8 * q:8 * q + 8]}) == 8


@pytest.mark.parametrize("B,HKV", [(8, 1), (8, 12), (16, 8), (32, 3)])
def test_scale_bytes_of_a_chunk(B, HKV):
    """The scale area: [K|V][16][Hkv] (halves of it from a 32-token block), or
    [block][K|V][8][Hkv] for two 8-token blocks; every copy 16-byte aligned."""
    pool = np.arange(4 * 2 * B * HKV).reshape(4, 2, B, HKV)
    flat = pool.reshape(-1)
    sb = 32 * HKV
    for ab in range(4):
        if B == 16:
            area = flat[2 * sb:3 * sb]
            src = [(2 * sb, sb)]
        elif B == 32:
            row = (ab & 1) * 16
            at = (2 * 64 + row) * HKV
            src = [(at, sb // 2), (at + 32 * HKV, sb // 2)]
            area = np.concatenate([flat[a:a + n] for a, n in src])
        else:
            src = [(3 * sb // 2, sb // 2), (1 * sb // 2, sb // 2)]
            area = np.concatenate([flat[a:a + n] for a, n in src])
        assert all(a % 16 == 0 and n % 16 == 0 for a, n in src)
        for hk in range(HKV):
            for j in range(16):
                kr = (j & 7) + 16 * (j >> 3) if B == 8 else j
                blk, off = (2, j) if B == 16 else (2, (ab & 1) * 16 + j) if B == 32 else ((3, 1)[j >> 3], j & 7)
                assert area[kr * HKV + hk] == pool[blk, 0, off, hk]
                assert area[(kr + (8 if B == 8 else 16)) * HKV + hk] == pool[blk, 1, off, hk]


@pytest.mark.parametrize("vec_per_row", [1, 2, 3, 5, 8, 24, 64, 100, 128, 192, 640, 1000, 4096, 5000, 1 << 20])
def test_words_are_split_into_tokens_exactly(vec_per_row):
    """row_split's reciprocal over every kind of word number below 2^31."""
    d = 2 * vec_per_row
    shift = (d - 1).bit_length()
    mul = ((((1 << shift) - d) << 32) // d) + 1
    assert mul < 1 << 32
    rng = np.random.default_rng(vec_per_row)
    w = np.concatenate([rng.integers(0, 1 << 31, 5000), np.arange(3 * d if d < 5000 else 3),
                        (1 << 31) - 1 - np.arange(min(3 * d, 5000)),
                        d * rng.integers(0, (1 << 31) // d, 500), d * rng.integers(1, (1 << 31) // d + 1, 500) - 1])
    w = w[(w >= 0) & (w < 1 << 31)].astype(np.uint64)
    total = ((np.uint64(mul) * w) >> np.uint64(32)) + w
    assert (total < 1 << 32).all()
    assert np.array_equal(total >> np.uint64(shift), w // np.uint64(d))


# ------------------------------------------------------------------ rows on the decode stream
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_few_rows(lib, group):
    few = lambda n: lib.pkv_quant_few_rows(n, 2 * group, 2)  # noqa: E731
    assert few(0) == few(1) == 1
    for n in range(1, 64 // group + 1):
        assert few(n) == n
    for n in (64 // group + 1, 512, 100000):
        assert few(n) == 8 // group
    assert few(-1) == E("PKV_ERR_BAD_SHAPE")
    assert lib.pkv_quant_few_rows(1, 3, 2) == E("PKV_ERR_BAD_SHAPE")
    assert lib.pkv_quant_few_rows(1, 6, 2) == E("PKV_ERR_UNSUPPORTED")
    assert lib.pkv_quant_few_rows(1, 4, 0) == E("PKV_ERR_BAD_SHAPE")


def test_options_of_the_rows(lib):
    def opt(**kw):
        o = binding.pkv_attention_options()
        for i, v in kw.items():
            o.reserved[int(i[1:])] = v
        return ctypes.pointer(o)

    for rows in (0, 1, 16, 32):  # 2 q heads per kv head; the next check decides
        assert _attn(lib, opt=opt(r1=rows), q=None) == E("PKV_ERR_NULL_POINTER")
    for bad in (dict(r1=-1), dict(r1=33), dict(r2=1), dict(r3=1), dict(r0=2)):
        # (without a GPU the device is asked for first)
        assert lib.pkv_quant_attention_workspace_size(4, 8, 4, _layout(), 0, opt(**bad)) < 0
        assert _attn(lib, opt=opt(**bad)) < 0
    assert binding._options(None, few_rows=3).contents.reserved[E("PKV_OPTIONS_FEW_ROWS")] == 3
    with pytest.raises(ValueError):
        binding.StepCalls(**{k: v for k, v in tensors().items() if k != "kv_scales"}, **SIZES, few_rows=2)


def test_chunk_keys(lib):
    assert binding.quant_chunk_keys([1, 1, 1], [100, 5, 17], 4, 16) == 0
    assert binding.quant_chunk_keys([5, 16, 1], [100, 50, 17], 4, 16) == 0  # 16 x 4 units
    assert binding.quant_chunk_keys([5, 17, 2], [100, 50, 17], 4, 16) == 112 + 64
    assert binding.quant_chunk_keys([], [], 4, 16) == 0
    assert binding.quant_chunk_keys([5, 17, 2], [100, 50, 17], 4, 16, few_rows=5) == 64


# ------------------------------------------------------------------ refusals of the C calls
def _write(lib, name="pkv_quant_kv_write", **kw):
    a = dict(kv=FAKE, sc=FAKE, k=FAKE, v=FAKE, ks=0, vs=0, slots=FAKE, T=4, lay=_layout())
    a.update(kw)
    if name == "pkv_quant_kv_read":
        return lib.pkv_quant_kv_read(a["k"], a["v"], a["ks"], a["vs"], a["kv"], a["sc"], a["slots"],
                                     a["T"], a["lay"], None)
    return lib.pkv_quant_kv_write(a["kv"], a["sc"], a["k"], a["v"], a["ks"], a["vs"], a["slots"],
                                  a["T"], a["lay"], None)


@pytest.mark.parametrize("name", ["pkv_quant_kv_write", "pkv_quant_kv_read"])
def test_row_calls_reject_bad_arguments(lib, name):
    W = lambda **kw: _write(lib, name, **kw)  # noqa: E731
    for bs in (4, 24, 64):
        assert W(lay=_layout(bs=bs)) == E("PKV_ERR_UNSUPPORTED")
    assert W(lay=_layout(bs=0)) == E("PKV_ERR_BAD_SHAPE")
    assert W(lay=_layout(d=96)) == E("PKV_ERR_UNSUPPORTED")
    assert W(lay=_layout(nb=0)) == E("PKV_ERR_BAD_SHAPE")
    assert W(T=-1) == E("PKV_ERR_BAD_SHAPE")
    assert W(ks=64) == E("PKV_ERR_BAD_SHAPE")
    assert W(vs=130) == E("PKV_ERR_MISALIGNED")
    for p in ("kv", "sc", "k", "v", "slots"):
        assert W(**{p: None}) == E("PKV_ERR_NULL_POINTER"), p
    for p in ("kv", "sc", "k", "v"):
        assert W(**{p: MISALIGNED}) == E("PKV_ERR_MISALIGNED"), p
    assert W(kv=None, sc=None, k=None, v=None, slots=None, T=0) == E("PKV_OK")


def test_mapped_write_rejects_bad_arguments(lib):
    def SW(**kw):
        a = dict(kv=FAKE, sc=FAKE, k=FAKE, v=FAKE, ks=0, vs=0, slots=FAKE, bt=FAKE, maxb=8, qsl=FAKE,
                 nc=FAKE, R=2, T=4, lay=_layout())
        a.update(kw)
        return lib.pkv_quant_slot_mapping_and_write(
            a["kv"], a["sc"], a["k"], a["v"], a["ks"], a["vs"], a["slots"], a["bt"], a["maxb"],
            a["qsl"], a["nc"], a["R"], a["T"], a["lay"], None)

    for kw in (dict(T=-1), dict(R=-1), dict(maxb=-1), dict(ks=64)):
        assert SW(**kw) == E("PKV_ERR_BAD_SHAPE"), kw
    for p in ("kv", "sc", "k", "v", "bt", "qsl", "nc"):
        assert SW(**{p: None}) == E("PKV_ERR_NULL_POINTER"), p
    assert SW(sc=MISALIGNED) == E("PKV_ERR_MISALIGNED")
    assert SW(lay=_layout(bs=12)) == E("PKV_ERR_UNSUPPORTED")
    assert SW(kv=None, sc=None, k=None, v=None, bt=None, qsl=None, nc=None, T=0) == E("PKV_OK")


def _attn(lib, write=False, **kw):
    a = dict(out=FAKE, q=FAKE, qs=0, kv=FAKE, sc=FAKE, k=FAKE, v=FAKE, ks=0, vs=0, slots=FAKE, bt=FAKE,
             maxb=8, sl=FAKE, qsl=FAKE, nc=FAKE, R=2, T=2, mq=1, ms=100, Hq=4, scale=0.125,
             lay=_layout(), ws=ctypes.c_void_p(0x10000), wsb=1 << 20, opt=None)
    a.update(kw)
    rows = [a[x] for x in ("k", "v", "ks", "vs", "slots")] if write else []
    f = lib.pkv_quant_paged_attention_with_write if write else lib.pkv_quant_paged_attention
    return f(a["out"], a["q"], a["qs"], a["kv"], a["sc"], *rows, a["bt"], a["maxb"], a["sl"], a["qsl"],
             a["nc"], a["R"], a["T"], a["mq"], a["ms"], a["Hq"], a["scale"], a["lay"], a["ws"],
             a["wsb"], a["opt"], None)


@pytest.mark.parametrize("write", [False, True])
def test_attention_rejects_bad_arguments(lib, write):
    A = lambda **kw: _attn(lib, write, **kw)  # noqa: E731
    for kw in (dict(Hq=3), dict(R=-1), dict(T=-1), dict(ms=200), dict(scale=0.0),
               dict(scale=float("nan")), dict(qs=100)):
        assert A(**kw) == E("PKV_ERR_BAD_SHAPE"), kw
    assert A(Hq=6) == E("PKV_ERR_UNSUPPORTED")
    assert A(lay=_layout(d=80)) == E("PKV_ERR_UNSUPPORTED")
    for p in ("out", "q", "kv", "sc", "bt", "sl", "qsl", "nc") + (("k", "v") if write else ()):
        assert A(**{p: None}) == E("PKV_ERR_NULL_POINTER"), p
    for p in ("out", "q", "kv", "sc") + (("k", "v") if write else ()):
        assert A(**{p: MISALIGNED}) == E("PKV_ERR_MISALIGNED"), p
    assert A(ws=None) == E("PKV_ERR_WORKSPACE")
    assert A(ws=ctypes.c_void_p(0x10010)) == E("PKV_ERR_WORKSPACE")
    if not write:
        assert A(R=0) == E("PKV_OK")


def test_copy_rejects_bad_arguments(lib):
    C = lib.pkv_quant_copy_blocks
    assert C(FAKE, FAKE, 4, FAKE, FAKE, 4, FAKE, 2, _layout(bs=48), None) == E("PKV_ERR_UNSUPPORTED")
    assert C(FAKE, FAKE, 0, FAKE, FAKE, 4, FAKE, 2, _layout(), None) == E("PKV_ERR_BAD_SHAPE")
    assert C(FAKE, FAKE, 4, FAKE, FAKE, 4, FAKE, -1, _layout(), None) == E("PKV_ERR_BAD_SHAPE")
    assert C(FAKE, None, 4, FAKE, FAKE, 4, FAKE, 2, _layout(), None) == E("PKV_ERR_NULL_POINTER")
    assert C(FAKE, FAKE, 4, FAKE, MISALIGNED, 4, FAKE, 2, _layout(), None) == E("PKV_ERR_MISALIGNED")
    assert C(None, None, 4, None, None, 4, None, 0, _layout(), None) == E("PKV_OK")


def test_workspace_size_rejects_bad_arguments(lib):
    S = lambda R=4, maxb=8, Hq=4, lay=_layout(), keys=0: lib.pkv_quant_attention_workspace_size(  # noqa: E731
        R, maxb, Hq, lay, keys, None)
    assert S(R=-1) == S(maxb=-1) == S(keys=-1) == S(Hq=3) == E("PKV_ERR_BAD_SHAPE")
    assert S(keys=1 << 30) == E("PKV_ERR_BAD_SHAPE")
    assert S(Hq=6) == S(lay=_layout(d=96)) == E("PKV_ERR_UNSUPPORTED")


# ------------------------------------------------------------------ refusals of the binding
class Stand:
    """What the binding asks of a CUDA tensor."""
    is_cuda = True

    def __init__(self, dtype, *shape, device=0, stride=None):
        self.dtype, self.shape, self.device = dtype, torch.Size(shape), torch.device("cuda", device)
        self._stride = stride

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        s = self._stride or tuple(self.shape[j + 1:].numel() for j in range(len(self.shape)))
        return s if i is None else s[i]

    def is_contiguous(self):
        return self._stride is None

    def is_pinned(self):
        return False

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 0x10000

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 1


class Calls:
    """A library that takes every call."""

    def __init__(self):
        self.names = []

    def __getattr__(self, name):
        def call(*args):
            self.names.append(name)
            return 1 if name == "pkv_quant_few_rows" else 0
        return call


T, HQ, HKV, D, R, NB, WIDTH = 5, 4, 2, 64, 3, 8, 4


def tensors(**kw):
    bf, i32 = torch.bfloat16, torch.int32
    out = dict(out=Stand(bf, T, HQ, D), q=Stand(bf, T, HQ, D),
               kv_cache=Stand(torch.float8_e4m3fn, NB, 2, 16, HKV, D),
               kv_scales=Stand(torch.uint8, NB, 2, 16, HKV), key=Stand(bf, T, HKV, D),
               value=Stand(bf, T, HKV, D), block_table=Stand(i32, R, WIDTH), seq_lens=Stand(i32, R),
               query_start_loc=Stand(i32, R + 1), num_computed_tokens=Stand(i32, R),
               workspace=Stand(torch.uint8, 512), slot_mapping=Stand(torch.int64, T))
    out.update(kw)
    return out


SIZES = dict(max_query_len=3, max_seq_len=60, scale=0.125)
BINDINGS = {
    "pkv_quant_kv_write": (binding.pkv_quant_kv_write, "kv_cache kv_scales key value slot_mapping", {}),
    "pkv_quant_kv_read": (binding.pkv_quant_kv_read, "key value kv_cache kv_scales slot_mapping", {}),
    "pkv_quant_slot_mapping_and_write": (
        binding.pkv_quant_slot_mapping_and_write,
        "kv_cache kv_scales key value block_table query_start_loc num_computed_tokens slot_mapping", {}),
    "pkv_quant_paged_attention": (
        binding.pkv_quant_paged_attention,
        "out q kv_cache kv_scales block_table seq_lens query_start_loc num_computed_tokens workspace", SIZES),
    "pkv_quant_paged_attention_with_write": (
        binding.pkv_quant_paged_attention_with_write,
        "out q kv_cache kv_scales key value block_table seq_lens query_start_loc num_computed_tokens "
        "workspace slot_mapping", SIZES),
    "StepCalls": (lambda **kw: binding.StepCalls(**kw).attend(),
                  "out q kv_cache kv_scales key value block_table seq_lens query_start_loc "
                  "num_computed_tokens workspace slot_mapping", SIZES),
}


@pytest.fixture
def library(monkeypatch):
    calls = Calls()
    monkeypatch.setattr(binding, "load", lambda *a, **k: calls)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(binding, "_current_stream", lambda device: 7)
    return calls


def _call(name, **kw):
    f, args, sizes = BINDINGS[name]
    t = tensors(**kw)
    return f(**{a: t[a] for a in args.split()}, **sizes)


@pytest.mark.parametrize("name", BINDINGS)
def test_binding_makes_the_call(library, name):
    _call(name)
    assert library.names == ["pkv_quant_paged_attention" if name == "StepCalls" else name]


@pytest.mark.parametrize("name", BINDINGS)
def test_binding_refuses_other_devices_types_and_shapes(library, name):
    f, args, _ = BINDINGS[name]
    good = tensors()
    for a in args.split():
        t = good[a]
        with pytest.raises(ValueError):  # another device than the pool's
            _call(name, **{a: Stand(t.dtype, *t.shape, device=1)})
        if a == "workspace":
            continue
        with pytest.raises(ValueError):
            _call(name, **{a: Stand(torch.float64, *t.shape)})
        if a not in ("block_table", "kv_cache"):
            with pytest.raises(ValueError):
                _call(name, **{a: Stand(t.dtype, t.shape[0] + 1, *t.shape[1:])})
    for a in ("q", "key", "value"):
        if a in args.split():
            h = good[a].shape[1]
            for stride in ((0, D, 1), (h * D, 2 * D, 1), (h * D, D, 2), (D, D, 1)):
                with pytest.raises(ValueError):
                    _call(name, **{a: Stand(torch.bfloat16, T, h, D, stride=stride)})
            with pytest.raises(ValueError):
                _call(name, **{a: Stand(torch.bfloat16, T, h, D // 2)})
    assert library.names == []


def test_binding_refuses_tensors_off_the_current_device(library, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for name in BINDINGS:
        with pytest.raises(ValueError):
            _call(name)
    assert library.names == []


def test_chunk_keys_of_a_longer_maximum(lib):
    """A call whose max_query_len is above the step's longest request expands more."""
    assert binding.quant_chunk_keys([5, 3, 1], [100, 50, 17], 4, 16) == 0
    assert binding.quant_chunk_keys([5, 3, 1], [100, 50, 17], 4, 16, max_query_len=16) == 0
    assert binding.quant_chunk_keys([5, 3, 1], [100, 50, 17], 4, 16, max_query_len=17) == 112 + 64
    assert binding.quant_chunk_keys([5, 3, 1], [100, 50, 17], 4, 16, few_rows=3, max_query_len=17) == 112


@pytest.mark.parametrize("name", ["pkv_quant_kv_write", "pkv_quant_kv_read"])
def test_scales_of_another_shape_are_refused(library, name):
    for shape in ((NB, 2, 16, HKV, 1), (NB, 2, 16), (NB, 2, 8, HKV), (NB, 1, 16, HKV), (NB, 2, 16, HKV + 1)):
        with pytest.raises(ValueError):
            _call(name, kv_scales=Stand(torch.uint8, *shape))
    assert library.names == []
