"""The operators around the recurrence where calls go wrong: streams of their own, states and
gradients beside infinities, sizes that a kernel's integers do not hold, paths that only large
calls take.  References are the definitions in 64 bits (layer_reference)."""
import pytest
import torch

import layer_reference as ref
import workloads
from conftest import cuda_ok
from test_layer_ops import DEV, DTYPES, NAMES, conv_inputs, norm_inputs, ok, same, scan_args, scan_inputs

gpu = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]


def gpu_test(f):
    for mark in gpu:
        f = mark(f)
    return f


# ---- a stream of the call's own ---------------------------------------------------------


def stream_calls(lib, seed=35):
    """Every entry point as a function of its stream that returns the tensors it made."""
    lengths = [700, 0, 33, 2000]
    cu = ref.offsets(lengths, DEV)
    c, cg = conv_inputs(torch.bfloat16, D=512, lengths=lengths, seed=seed)
    s, sg = scan_inputs(torch.bfloat16, D=512, lengths=lengths, seed=seed)
    n, ndy = norm_inputs(torch.bfloat16, 3003, 512, gate=True, seed=seed)

    conv = (c["x"], c["weight"], c["bias"], c["h0"], cu)
    r = workloads.to_device(workloads.make_inputs(1, 0, 2, 4, 128, 128, gate_mu=3.0, h0=True, seed=seed,
                                                  lengths=lengths), DEV)
    do, dht = torch.randn_like(r["v"]), torch.randn_like(r["h0"])
    rec = [r[k] for k in ("q", "k", "v", "beta", "g", "h0", "cu_seqlens")]
    calls = dict(
        chunk_fwd=lambda st: lib.chunk_fwd(*rec, stream=st),
        recurrent_fwd=lambda st: lib.recurrent_fwd(*rec, stream=st),
        chunk_bwd=lambda st: lib.chunk_bwd(*rec, do=do, dht=dht, stream=st),
        causal_conv_fwd=lambda st: lib.causal_conv_fwd(*conv, stream=st),
        causal_conv_bwd=lambda st: lib.causal_conv_bwd(*conv, dy=cg["dy"], dht=cg["dht"], stream=st),
        selective_scan_fwd=lambda st: lib.selective_scan_fwd(*scan_args(s), cu, stream=st),
        selective_scan_bwd=lambda st: lib.selective_scan_bwd(*scan_args(s), cu, dy=sg["dy"], dht=sg["dht"], stream=st),
        layer_norm_fwd=lambda st: [lib.layer_norm_fwd(n["x"], n["weight"], n["bias"], n["z"], stream=st)],
        layer_norm_bwd=lambda st: lib.layer_norm_bwd(n["x"], n["weight"], n["bias"], n["z"], dy=ndy, stream=st))
    return {k: (lambda st, f=f: outputs(f(st))) for k, f in calls.items()}


def outputs(o):
    return [v for v in (o.values() if isinstance(o, dict) else o) if v is not None]


CALLS = ("chunk_fwd", "recurrent_fwd", "chunk_bwd", "causal_conv_fwd", "causal_conv_bwd", "selective_scan_fwd",
         "selective_scan_bwd", "layer_norm_fwd", "layer_norm_bwd")


def agree(name, got, want):
    """Bit for bit; the recurrence's backward adds atomically and is held to its bound, 5e-3 of the norm."""
    if name != "chunk_bwd":
        return same(got, want)
    return len(got) == len(want) and all((a - b).norm() <= 5e-3 * b.norm() for a, b in zip(got, want))


def stream_of(tensor):
    """Handle of the stream whose memory a tensor lies in."""
    at = tensor.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= at < s["address"] + s["total_size"])


def reserved(handle):
    return sum(s["total_size"] for s in torch.cuda.memory_snapshot() if s["stream"] == handle)


@gpu_test
@pytest.mark.parametrize("name", CALLS)
def test_what_a_call_allocates_is_its_streams(lib, name):
    """Outputs and workspace come from the memory of the stream that the call was given."""
    call = stream_calls(lib)[name]
    side = torch.cuda.Stream()
    here = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        torch.cuda.empty_cache()
        before = reserved(here)
        outs = call(stream)
        assert [stream_of(o) for o in outs] == [side.cuda_stream] * len(outs)
        assert reserved(here) == before
        side.synchronize()
    assert all(stream_of(o) == here for o in call(None))
    torch.cuda.synchronize()
    ok(lib)


@gpu_test
@pytest.mark.parametrize("name", CALLS)
def test_calls_on_a_stream_beside_another(lib, name):
    """Neither memory that the current stream gave back while its work on it waits, nor outputs dropped
    while the call has yet to run, pass between the two streams."""
    call = stream_calls(lib)[name]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        # what the current stream will read only later, given back at once
        held = [torch.full_like(w, 3.0) for w in want for _ in range(2)]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        later = [h.clone() for h in held]
        del held
        got = call(stream)
        torch.cuda.synchronize()
        assert all((v == 3).all() for v in later)
        assert agree(name, got, want)
        # outputs dropped before the call has run
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        del got
        got = call(stream)[:1]
        mine = [torch.full_like(w, 5.0) for w in want for _ in range(2)]
        torch.cuda.synchronize()
        assert all((v == 5).all() for v in mine)
        assert agree(name, got, want[:1])
    ok(lib)


@gpu_test
def test_calls_given_the_default_stream(lib):
    """The default stream by its handle, 0 or 1, from under another stream."""
    calls = stream_calls(lib)
    want = {k: f(None) for k, f in calls.items()}
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = [{k: f(handle) for k, f in calls.items()} for handle in (0, 1)]
    torch.cuda.synchronize()
    for g in got:
        for k in want:
            assert agree(k, g[k], want[k]), k
            assert all(stream_of(o) == 0 for o in g[k])


@gpu_test
@pytest.mark.parametrize("name", CALLS)
def test_calls_given_a_stream_that_is_captured(lib, name):
    """The capturing stream as an argument, by object and by handle: replays give the call's results."""
    call = stream_calls(lib)[name]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                held = call(stream)
        for _ in range(2):
            for h in held:
                h.fill_(7)
            graph.replay()
            torch.cuda.synchronize()
            assert agree(name, held, want)
    ok(lib)


# ---- infinities -----------------------------------------------------------------------------


@gpu_test
@pytest.mark.parametrize("lengths", [[21], [24], [1, 9, 16, 30], [131], [0, 70, 3]])
@pytest.mark.parametrize("N", [16, 64])
def test_scan_gradient_of_the_rates_beside_an_overflow(lib, lengths, N):
    """The last token's state overflows fp32 in one channel.  d_A takes the states before a token alone, and
    those are finite: it is what it is in 64 bits, whether or not the length fills the kernel's pieces."""
    t, grads = scan_inputs(torch.float32, D=12, N=N, lengths=lengths, gate=False, seed=15)
    t["dt"], t["dt_bias"] = t["dt"].abs() * 0.2 + 0.05, None
    at, n = 0, []
    for length in lengths:
        if length:
            last = at + length - 1
            t["dt"][0, last], t["B"][0, last], t["x"][0, last, 3] = 1.0, 4.0, 2e38
            n.append(last)
        at += length
    grads["dy"][0, n] *= 1e-3
    cu = ref.offsets(lengths, DEV)
    y, ht = lib.selective_scan_fwd(*scan_args(t), cu, dt_softplus=False)
    assert all(torch.isinf(ht[i, 3]).all() for i, length in enumerate(lengths) if length)
    out = lib.selective_scan_bwd(*scan_args(t), cu, dt_softplus=False, dy=grads["dy"])
    ok(lib)
    leaves = ref.in_64_bits(t, grad=True)
    y64, ht64 = ref.scan(leaves, lengths, softplus=False)
    want = ref.gradients([y64, ht64], [grads["dy"], None], leaves)["A"]
    # roundings of test_layer_ops.scan_check
    ref.close(out["dA"], want, 30 * max(lengths) + 64 + sum(lengths), "dA")


@gpu_test
@pytest.mark.parametrize("lengths", [[200], [40, 333, 0, 75], [1000]])
def test_scan_infinite_state_stays_infinite_over_chunks(lib, lengths):
    """Each token's decay is e^-6, a chunk's lies below what fp32 holds: an infinite state decays to
    an infinite one all the same."""
    t, _ = scan_inputs(torch.float32, D=7, lengths=lengths, gate=False, seed=16)
    t["dt"], t["dt_bias"], t["A"] = torch.full_like(t["dt"], 2.0), None, torch.full_like(t["A"], -3.0)
    at = 0
    for length in lengths:
        if length:
            t["x"][0, at + 5, 3] = float("inf")
        at += length
    cu = ref.offsets(lengths, DEV)
    assert lib.load().dn_selective_scan_fwd_workspace_bytes(len(lengths), 1, sum(lengths), 7, 1, 16, lib.DN_F32) > 0
    y64, ht64 = ref.scan(ref.in_64_bits(t), lengths, softplus=False)
    y, ht = lib.selective_scan_fwd(*scan_args(t), cu, dt_softplus=False)
    ok(lib)
    for n, length in enumerate(lengths):
        if length:
            assert torch.isinf(ht64[n, 3]).all()
            assert torch.equal(ht[n, 3].double().cpu(), ht64[n, 3])
    keep = [d for d in range(7) if d != 3]
    ref.close(y[:, :, keep], y64[:, :, keep], 10 * max(lengths) + 64, "y of the others")
    ref.close(ht[:, keep], ht64[:, keep], 10 * max(lengths) + 64, "ht of the others")


@gpu_test
@pytest.mark.parametrize("T", [1, 2, 33, 200])
@pytest.mark.parametrize("G", [1, 2])
def test_scan_without_d_has_no_such_term(lib, T, G):
    """D absent: an infinite input gives what C h gives, not a NaN of 0 times infinity; the same in a prompt
    and in a single token, and in the gradient of the gate."""
    t, grads = scan_inputs(torch.float32, B=2, T=T, D=2 * 3 * G, G=G, extras=False, seed=17)
    t["B"], t["C"], t["z"] = t["B"].abs() + 0.1, t["C"].abs() + 0.1, t["z"].abs() + 0.1
    t["x"][1, T - 1, 4] = float("inf")
    y64, ht64 = ref.scan(ref.in_64_bits(t))
    y, ht = lib.selective_scan_fwd(*scan_args(t))
    out = lib.selective_scan_bwd(*scan_args(t), dy=grads["dy"])
    ok(lib)
    assert y64[1, T - 1, 4] == float("inf") and y[1, T - 1, 4] == float("inf")
    assert torch.isinf(ht[1, 4]).all()
    assert torch.isinf(out["dz"][1, T - 1, 4])
    keep = [d for d in range(t["x"].shape[2]) if d != 4]
    ref.close(y[:, :, keep], y64[:, :, keep], 10 * T + 64, "y of the others")


@gpu_test
@pytest.mark.parametrize("T", [100, 333])
def test_scan_growing_rates(lib, T):
    """Rates above zero: a chunk's growth passes what fp32 holds while nothing is there to grow (no input
    before the last tokens, no gradient behind the first).  Nothing stays nothing, in states and gradients."""
    t, grads = scan_inputs(torch.float32, B=1, T=T, D=9, gate=True, h0=False, seed=18)
    t["dt"], t["dt_bias"] = torch.full_like(t["dt"], 1.0), None
    t["A"] = torch.full_like(t["A"], 6.0 if T == 100 else 2.0)
    t["x"][:, :T - 8] = 0
    grads["dy"][:, 8:] = 0
    y64, ht64 = ref.scan(leaves := ref.in_64_bits(t, grad=True), softplus=False)
    y, ht = lib.selective_scan_fwd(*scan_args(t), dt_softplus=False)
    ref.close(y, y64, 10 * T + 64, "y")
    ref.close(ht, ht64, 10 * T + 64, "ht")
    out = lib.selective_scan_bwd(*scan_args(t), dt_softplus=False, dy=grads["dy"])
    ok(lib)
    want = ref.gradients([y64], [grads["dy"]], leaves)
    for name in NAMES:
        if t[name] is not None:
            ref.close(out["d" + name], want[name], 30 * T + 64, "d" + name)


@gpu_test
def test_scan_small_gradient_grows_past_a_chunk_s_factor(lib):
    """A gradient of 1e-30 eleven tokens on, rates of e^9: the product of the rates passes fp32, the gradient
    at the first token does not."""
    t, grads = scan_inputs(torch.float32, B=1, T=40, D=9, gate=False, h0=True, extras=False, seed=19)
    t["dt"], t["A"] = torch.full_like(t["dt"], 1.0), torch.full_like(t["A"], 9.0)
    t["x"][:] = 0
    t["h0"][:] = 0
    grads["dy"][:] = 0
    grads["dy"][0, 11] = 1e-30
    out = lib.selective_scan_bwd(*scan_args(t), dt_softplus=False, dy=grads["dy"])
    ok(lib)
    leaves = ref.in_64_bits(t, grad=True)
    y64, _ = ref.scan(leaves, softplus=False)
    want = ref.gradients([y64], [grads["dy"]], leaves)
    for name in ("x", "h0"):
        ref.close(out["d" + name], want[name], 30 * 40 + 64, "d" + name)


# ---- what the library says of a call, and what it refuses --------------------------------------


@gpu_test
@pytest.mark.parametrize("dtype,short", [(torch.bfloat16, "bf16"), (torch.float32, "f32")])
def test_last_kernel_tells_the_path(lib, dtype, short):
    """dn_last_kernel names the kernels that a call launched: single tokens, whole sequences, chunks."""
    for T, conv, scan in ((1, "conv_step", "scan_step"), (20, "conv_fwd", "scan_fwd"),
                          (500, "conv_fwd", "scan_state+scan_combine+scan_fwd")):
        c, _ = conv_inputs(dtype, B=2, T=T, D=24, seed=1)
        lib.causal_conv_fwd(c["x"], c["weight"], c["bias"], c["h0"])
        assert lib.dn_last_kernel() == "%s<%s>" % (conv, short)
        s, _ = scan_inputs(dtype, B=2, T=T, D=24, seed=1)
        lib.selective_scan_fwd(*scan_args(s))
        assert lib.dn_last_kernel() == "%s<%s>" % (scan, short)
        lib.causal_conv_bwd(c["x"], c["weight"], c["bias"], c["h0"], dy=c["x"])
        assert lib.dn_last_kernel() == "conv_bwd+conv_bwd_sums<%s>" % short
        lib.selective_scan_bwd(*scan_args(s), dy=s["x"])
        assert lib.dn_last_kernel() == "scan_bwd_state+scan_combine+scan_bwd+scan_bwd_bc+scan_bwd_sums<%s>" % short
    n, dy = norm_inputs(dtype, 5, 24, seed=1)
    lib.layer_norm_fwd(n["x"], n["weight"])
    assert lib.dn_last_kernel() == "norm_fwd<%s>" % short
    lib.layer_norm_bwd(n["x"], n["weight"], dy=dy)
    assert lib.dn_last_kernel() == "norm_bwd+norm_bwd_sums<%s>" % short
    lib.layer_norm_bwd(n["x"], dy=dy)
    assert lib.dn_last_kernel() == "norm_bwd<%s>" % short
    cu = ref.offsets([1, 1], DEV)  # offsets are on the device: these tokens are not known to be single ones
    lib.causal_conv_fwd(c["x"][:1, :2].contiguous(), c["weight"], c["bias"], c["h0"], cu)
    assert lib.dn_last_kernel() == "conv_fwd<%s>" % short
    ok(lib)


@pytest.mark.parametrize("shape", [(1, 2**32 + 3, 1), (2**32 + 2, 1, 1), (1, 1, 2**32 + 8)])
def test_sizes_above_an_int_are_refused(monkeypatch, shape):
    """A size that the C arguments cannot hold is an error, not another size (tensors without memory)."""
    import chunkwise_gated_delta_chunk_gb300 as dn
    monkeypatch.setattr(dn, "_device_of", lambda x, torch: x.device)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)

    def empty(*s):
        return torch.empty(s, device="meta")

    B, T, D = shape
    x = empty(*shape)
    calls = [lambda: dn.causal_conv_fwd(x, empty(D, 4)), lambda: dn.causal_conv_bwd(x, empty(D, 4), dy=x),
             lambda: dn.selective_scan_fwd(x, x, empty(D, 16), empty(B, T, 1, 16), empty(B, T, 1, 16)),
             lambda: dn.selective_scan_bwd(x, x, empty(D, 16), empty(B, T, 1, 16), empty(B, T, 1, 16), dy=x)]
    if D > 1:
        calls += [lambda: dn.layer_norm_fwd(x), lambda: dn.layer_norm_bwd(x, dy=x)]
    for call in calls:
        with pytest.raises(dn.DnError) as e:
            call()
        assert e.value.status == dn.DN_ERR_UNSUPPORTED


def test_more_sequences_than_an_int_are_refused(monkeypatch):
    import chunkwise_gated_delta_chunk_gb300 as dn
    monkeypatch.setattr(dn, "_device_of", lambda x, torch: x.device)
    x, cu = torch.empty(1, 8, 8, device="meta"), torch.empty(2**32 + 2, dtype=torch.int64, device="meta")
    with pytest.raises(dn.DnError) as e:
        dn.causal_conv_fwd(x, torch.empty(8, 4, device="meta"), cu_seqlens=cu, output_final_state=False)
    assert e.value.status == dn.DN_ERR_UNSUPPORTED
