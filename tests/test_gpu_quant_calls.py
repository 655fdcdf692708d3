"""How the 8-bit pool's calls are used together and beside one another: streams,
graphs, pools past 4 GB, a served sequence from its prompt to its last token."""

import numpy as np
import pytest

import oracle
from parity import bits_to_f64
from quant_cases import expected, quantised_step
from test_gpu_quant import E4M3, assert_within, host

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_hkv_gb300 import binding  # noqa: E402
from paged_kv_cache_hkv_gb300.runner import DeviceStep, bf16_to_numpy  # noqa: E402
from paged_kv_cache_hkv_gb300.synth import RequestSpec, make_step  # noqa: E402


@pytest.fixture(autouse=True)
def _clear_errors():
    binding.pkv_get_device_errors(clear=True)
    yield


STEPS = {
    "decode": [RequestSpec(700, 1), RequestSpec(20, 1), RequestSpec(3000, 1)],
    "few": [RequestSpec(700, 4), RequestSpec(20, 2), RequestSpec(1500, 3)],
    "mixed": [RequestSpec(300, 70), RequestSpec(20, 1), RequestSpec(800, 2)],
}


def steps(seed=0):
    return [make_step(specs, num_q_heads=16, num_kv_heads=4, head_dim=128, seed=seed + i)
            for i, specs in enumerate(STEPS.values())]


def test_calls_on_two_streams_at_once():
    """Each with its own buffers and workspace, on streams other than the current one."""
    made = steps()
    ready = [DeviceStep(s, quantised=True, write_in_attention=True) for s in made]
    want = [expected(s, quantised_step(s)[2]) for s in made]
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    for _ in range(20):
        for ds, stream in zip(ready, streams):
            ds.run(stream=stream)
    torch.cuda.synchronize()
    for ds, w in zip(ready, want):
        assert_within(ds.out_host(), *w)
    assert binding.pkv_get_device_errors(clear=True) == 0


def test_two_graphs_on_one_workspace():
    made = steps(5)
    ready = [DeviceStep(s, quantised=True, write_in_attention=True) for s in made]
    size = max(ds.workspace.numel() for ds in ready)
    workspace = torch.empty(size, dtype=torch.uint8, device="cuda")
    want = [expected(s, quantised_step(s)[2]) for s in made]
    graphs = []
    side = torch.cuda.Stream()
    for ds in ready:
        ds.workspace = workspace
        with torch.cuda.stream(side):
            ds.run()
            side.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                ds.run()
    for order in ((0, 1, 2), (2, 0, 1, 1, 0, 2)):
        for ds in ready:
            ds.out.fill_(5.0)
        workspace.fill_(255)  # nothing of it has to last from call to call
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for ds, w in zip(ready, want):
            assert_within(ds.out_host(), *w)
    assert binding.pkv_get_device_errors(clear=True) == 0


@pytest.mark.parametrize("scores", [{}, {"softcap": 20.0}])
def test_a_call_leaves_nothing_behind(scores):
    """The same step again after others: the same bits, whatever the workspace holds."""
    made = steps(9)
    ready = [DeviceStep(s, quantised=True, write_in_attention=True, **scores) for s in made]
    first = []
    for ds in ready:
        ds.run()
        first.append(ds.out_host())
    for fill in (0, 255, 127):
        for ds, f in zip(ready, first):
            ds.workspace.fill_(fill)
            ds.out.zero_()
            ds.run()
            assert np.array_equal(ds.out_host(), f)


def test_blocks_behind_four_gigabytes():
    B, hkv, hq, d, nb = 16, 8, 32, 128, 150_000  # 4.9 GB of codes
    codes = torch.zeros(nb, 2, B, hkv, d, dtype=torch.uint8, device="cuda").view(E4M3)
    scales = torch.full((nb, 2, B, hkv), 127, dtype=torch.uint8, device="cuda")
    lens, new = [200, 130, 90], [1, 3, 40]  # cached and new tokens
    T = sum(new)
    table = torch.full((3, 16), -1, dtype=torch.int32)
    ids = nb - 1 - 7 * np.arange(48)
    at = 0
    for r in range(3):
        n = -(-(lens[r] + new[r]) // B)
        table[r, :n] = torch.from_numpy(ids[at:at + n].astype(np.int32))
        at += n
    g = torch.Generator(device="cuda").manual_seed(3)
    rows = sum(lens)
    k, v = (torch.randn(rows + T, hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(T, hq, d, generator=g, device="cuda").bfloat16()
    slots = torch.cat([table[r, :].long().repeat_interleave(B)[:lens[r]] * B + torch.arange(lens[r]) % B
                       for r in range(3)]).cuda()
    binding.pkv_quant_kv_write(codes, scales, k[:rows], v[:rows], slots)
    back = [torch.empty_like(k[:rows]) for _ in range(2)]
    binding.pkv_quant_kv_read(*back, codes, scales, slots)
    for x, y in zip((k, v), back):
        c, s = oracle.quantise_rows(bf16_to_numpy(x[:rows]))
        assert np.array_equal(oracle.quant_pool_bits(c, s), bf16_to_numpy(y))
    i32 = dict(dtype=torch.int32, device="cuda")
    total = [a + b for a, b in zip(lens, new)]
    qsl = torch.tensor(np.concatenate([[0], np.cumsum(new)]), **i32)
    out = torch.empty_like(q)
    ws = torch.empty(binding.pkv_quant_attention_workspace_size(
        3, hq, codes, max_blocks_per_req=16, chunk_keys=binding.quant_chunk_keys(new, total, 4, B)),
        dtype=torch.uint8, device="cuda")
    binding.pkv_quant_paged_attention_with_write(
        out, q, codes, scales, k[rows:], v[rows:], table.cuda(), torch.tensor(total, **i32), qsl,
        torch.tensor(lens, **i32), max_query_len=max(new), max_seq_len=max(total), scale=d ** -0.5,
        workspace=ws)
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == 0
    # the same over a small pool of the used blocks
    used = sorted(int(b) for b in table.flatten() if b >= 0)
    small = torch.full_like(table, -1)
    for i, b in enumerate(used):
        small[table == b] = i
    pool = oracle.quant_pool_bits(host(codes[used]), scales[used].cpu().numpy())
    want, bound = oracle.scored_attention(bf16_to_numpy(q), pool, small.numpy(), total,
                                          qsl.cpu().numpy(), lens, d ** -0.5)
    assert_within(bf16_to_numpy(out), want, bound * 1.01)


def test_a_sequence_served_from_prompt_to_last_token():
    """A prompt in two chunks, tokens one by one, guesses of four, the blocks copied
    into another pool, the rows read back: the attention of every step against the
    oracle over what was written."""
    B, hkv, hq, d, nb = 16, 2, 8, 64, 40
    rng = np.random.default_rng(2)
    plan = [(0, 130), (130, 70)] + [(200 + i, 1) for i in range(18)] + [(218, 4), (222, 4), (226, 1)]
    total = plan[-1][0] + plan[-1][1]
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v, q = (torch.randn(total, h, d, generator=g, device="cuda").bfloat16() for h in (hkv, hkv, hq))
    table = torch.from_numpy(rng.permutation(nb)[:-(-total // B)].astype(np.int32)).cuda().view(1, -1)
    codes = torch.zeros(nb, 2, B, hkv, d, dtype=torch.uint8, device="cuda").view(E4M3)
    scales = torch.zeros(nb, 2, B, hkv, dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    ws = torch.empty(binding.pkv_quant_attention_workspace_size(
        1, hq, codes, max_blocks_per_req=table.shape[1], chunk_keys=total + B), dtype=torch.uint8,
        device="cuda")
    want_c, want_s = host(codes).copy(), scales.cpu().numpy().copy()
    kb, vb = bf16_to_numpy(k), bf16_to_numpy(v)
    for c, n in plan:
        if c == 210:  # swapped to another pool and on from there
            other = (torch.zeros_like(codes.view(torch.uint8)).view(E4M3), torch.zeros_like(scales))
            pairs = torch.stack([table[0], table[0].flip(0)], 1).contiguous()
            binding.pkv_quant_copy_blocks(*other, codes, scales, pairs)
            moved = table.flip(1).contiguous()
            order = table[0].cpu().numpy()
            new_c, new_s = np.zeros_like(want_c), np.zeros_like(want_s)
            new_c[order[::-1]], new_s[order[::-1]] = want_c[order], want_s[order]
            (codes, scales), table, want_c, want_s = other, moved, new_c, new_s
        slots = torch.empty(n, dtype=torch.int64, device="cuda")
        out = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
        binding.pkv_quant_paged_attention_with_write(
            out, q[c:c + n], codes, scales, k[c:c + n], v[c:c + n], table, torch.tensor([c + n], **i32),
            torch.tensor([0, n], **i32), torch.tensor([c], **i32), max_query_len=n, max_seq_len=c + n,
            scale=0.125, workspace=ws, slot_mapping=slots)
        want_c, want_s = oracle.quant_write(want_c, want_s, kb[c:c + n], vb[c:c + n], slots.cpu().numpy())
        pool = oracle.quant_pool_bits(want_c, want_s)
        ref, bound = oracle.scored_attention(bf16_to_numpy(q[c:c + n]), pool, table.cpu().numpy(), [c + n],
                                             [0, n], [c], 0.125)
        assert_within(bf16_to_numpy(out), ref, bound * 1.01, what=f"{n} tokens at {c}")
    assert np.array_equal(host(codes), want_c) and np.array_equal(scales.cpu().numpy(), want_s)
    slots = table[0].long().repeat_interleave(B)[:total] * B + torch.arange(total, device="cuda") % B
    back = [torch.empty_like(k) for _ in range(2)]
    binding.pkv_quant_kv_read(*back, codes, scales, slots)
    for x, y in zip((kb, vb), back):
        x, y = bits_to_f64(x), bits_to_f64(bf16_to_numpy(y))
        # half a step: 2^-4 of the value, or 2^-10 2^e where codes are subnormal, and the
        # row's largest is above 224 2^e: less than 2^-17 of it
        assert (np.abs(x - y) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -17 * np.abs(x).max(-1, keepdims=True)).all()
    assert binding.pkv_get_device_errors(clear=True) == 0


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (32, 8, 128)])
def test_q_and_v_of_any_size(hq, hkv, d):
    """Rows of q, K and V from tiny to huge (V's scales go into the weights' exponent,
    q and K's into the scores): the result keeps its relative accuracy, row by row."""
    rng = np.random.default_rng(d)
    specs = [RequestSpec(300, 1), RequestSpec(77, 3), RequestSpec(1000, 1)]
    step = make_step(specs, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, seed=8)

    def scaled(bits, size):
        x = bits_to_f64(bits) * size
        return bf16_to_numpy(torch.from_numpy(x.astype(np.float32)).bfloat16())

    vsize = 2.0 ** rng.integers(-60, 40, size=step.kv_cache.shape[0])[:, None, None, None]
    step.kv_cache = step.kv_cache.copy()
    step.kv_cache[:, 1] = scaled(step.kv_cache[:, 1], vsize)
    step.v = scaled(step.v, 2.0 ** -70)
    step.kv_cache[:, 0] = scaled(step.kv_cache[:, 0], 2.0 ** 30)
    step.k = scaled(step.k, 2.0 ** 30)
    step.q = scaled(step.q, 2.0 ** -30)
    ds = DeviceStep(step, quantised=True, write_in_attention=True)
    ds.run()
    ref, bound = expected(step, quantised_step(step)[2])
    assert_within(ds.out_host(), ref, bound)
    assert binding.pkv_get_device_errors(clear=True) == 0


def test_traced_calls():
    for step in steps(3):
        ds = DeviceStep(step, quantised=True)
        ds.slot_map_and_write()
        events = [torch.cuda.Event(enable_timing=True) for _ in range(binding.PKV_TRACE_EVENTS)]
        for e in events:
            e.record()
        binding.pkv_quant_paged_attention(
            ds.out, ds.q, ds.kv_cache, ds.kv_scales, ds.block_table, ds.seq_lens, ds.query_start_loc,
            ds.num_computed, max_query_len=step.max_query_len, max_seq_len=step.max_seq_len,
            scale=step.scale, workspace=ds.workspace, trace_events=events)
        torch.cuda.synchronize()
        assert all(a.elapsed_time(b) > 0 for a, b in zip(events, events[1:]))
        assert_within(ds.out_host(), *expected(step, quantised_step(step)[2]))


def test_values_of_nothing():
    """All V rows zero, and all K rows zero: outputs 0, and the mean of V."""
    step = make_step([RequestSpec(200, 1), RequestSpec(33, 4), RequestSpec(60, 40)], num_q_heads=8,
                     num_kv_heads=2, head_dim=128, seed=1)
    zero = np.zeros_like
    for which in (0, 1):
        step.kv_cache = step.kv_cache.copy()
        keep = step.kv_cache.copy()
        step.kv_cache[:, which] = 0
        k, v = step.k, step.v
        if which == 0:
            step.k = zero(k)
        else:
            step.v = zero(v)
        ds = DeviceStep(step, quantised=True, write_in_attention=True)
        ds.run()
        ref, bound = expected(step, quantised_step(step)[2])
        assert_within(ds.out_host(), ref, bound)
        if which == 1:
            assert not bits_to_f64(ds.out_host()).any()
        step.kv_cache, step.k, step.v = keep, k, v
