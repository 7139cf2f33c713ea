"""Device-side plumbing around the C ABI: torch allocates the inputs and
weights and provides the stream; every step of the FFN path runs in the
library's kernels (combine_peer_slot_gb300/afd.py)."""
import numpy as np

from . import afd as A
from . import workloads as W


class DeviceBytes:
    """Zero-copy uint8 view of a device allocation owned by the library, for
    inspecting or editing slot bytes from torch."""

    def __init__(self, ptr, nbytes):
        self.__cuda_array_interface__ = {"shape": (int(nbytes),), "typestr": "|u1",
                                         "data": (int(ptr), False), "version": 2}


def device_view(ptr, nbytes):
    import torch
    return torch.as_tensor(DeviceBytes(ptr, nbytes), device="cuda")


def act_tensor(a, act, device):
    """numpy activation storage (uint16 bf16 bits / float32) -> torch tensor."""
    import torch
    if act == "bf16":
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16).to(device)
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device)


class Runner:
    """One library context bound to a workload: inputs on the device, the
    layer weights registered, and helpers for pack / forward / unpack."""

    def __init__(self, w: W.Workload, gemm=A.AFD_GEMM_TENSOR, layers=None, stream=None,
                 max_total_tokens=0, wait_timeout_ns=0, device="cuda", flags=0, ring_depth=1,
                 canary=False):
        import torch
        self.w = w
        self.device = device
        self.layers = w.layers if layers is None else layers
        self.stream = stream if stream is not None else torch.cuda.current_stream()
        self.cfg = A.make_config(w.num_peers, w.token_cap, w.hidden, w.num_experts, w.topk,
                                 w.inter, w.shared_inter, act=w.act, renorm=w.renorm,
                                 routed_scaling=w.routed_scaling, max_layers=self.layers,
                                 max_total_tokens=max_total_tokens, gemm=gemm,
                                 wait_timeout_ns=wait_timeout_ns,
                                 flags=flags | (A.AFD_CFG_CANARY if canary else 0),
                                 ring_depth=ring_depth)
        self.ctx = A.afd_create(self.cfg, self.stream.cuda_stream)
        self.layout = A.afd_slot_layout(self.cfg)
        self.canary = bool(canary)
        self.host = W.host_inputs(w)
        self.x = [act_tensor(a, w.act, device) for a in self.host["x"]]
        self.Wg = torch.from_numpy(self.host["Wg"]).to(device)
        self.bias = None if self.host["bias"] is None else torch.from_numpy(self.host["bias"]).to(device)
        self.weights = []
        for layer in range(self.layers):
            wt = W.expert_weights(w, layer, device)
            self.weights.append(wt)
            A.afd_set_layer(self.ctx, layer, self.Wg.data_ptr(),
                            self.bias.data_ptr() if self.bias is not None else 0,
                            wt["W13"].data_ptr(), wt["Wd"].data_ptr(),
                            wt["W13s"].data_ptr() if wt["W13s"] is not None else 0,
                            wt["Wds"].data_ptr() if wt["Wds"] is not None else 0)
        self.seq = 0
        self.last_seq = {}
        dt = torch.bfloat16 if w.act == "bf16" else torch.float32
        self.out = [torch.empty((max(n, 1), w.hidden), dtype=dt, device=device) for n in w.seq_lens]
        self.batched = True  # pack / unpack all listed peers in one call (afd_pack_slots / afd_unpack_splits)

    # -- attention side, simulated ------------------------------------------------
    def pack_all(self, layer=0, stage=0, peers=None, with_shared=None):
        ws = (self.w.shared_inter > 0) if with_shared is None else with_shared
        peers = list(range(self.w.num_peers)) if peers is None else list(peers)
        if self.batched:
            seqs = [self.seq + 1 + i for i in range(len(peers))]
            ns = [self.w.seq_lens[p] for p in peers]
            rc = A.afd_pack_slots(self.ctx, peers, stage, layer,
                                  [self.x[p].data_ptr() if n else 0 for p, n in zip(peers, ns)], ns, ws, seqs)
            if rc:
                raise A.AfdError(rc, "afd_pack_slots")
            self.seq += len(peers)
            for p, s in zip(peers, seqs):
                self.last_seq[(p, stage)] = s
            return
        for p in peers:
            self.seq += 1
            n = self.w.seq_lens[p]
            rc = A.afd_pack_slot(self.ctx, p, stage, layer, self.x[p].data_ptr() if n else 0, n,
                                 ws, self.seq)
            if rc:
                raise A.AfdError(rc, "afd_pack_slot")
            self.last_seq[(p, stage)] = self.seq

    def forward(self, layer=0, stage=0, slots=None):
        slots = list(range(self.w.num_peers)) if slots is None else list(slots)
        lens = [self.w.seq_lens[p] for p in slots]
        return A.afd_ffn_forward(self.ctx, layer, stage, lens, slots)

    def unpack_all(self, stage=0, peers=None):
        peers = list(range(self.w.num_peers)) if peers is None else list(peers)
        if self.batched:
            ns = [self.w.seq_lens[p] for p in peers]
            rc = A.afd_unpack_splits(self.ctx, peers, stage,
                                     [self.out[p].data_ptr() if n else 0 for p, n in zip(peers, ns)], ns,
                                     [self.last_seq[(p, stage)] for p in peers])
            if rc:
                raise A.AfdError(rc, "afd_unpack_splits")
            return self.out
        for p in peers:
            n = self.w.seq_lens[p]
            rc = A.afd_unpack_split(self.ctx, p, stage, self.out[p].data_ptr() if n else 0, n,
                                    self.last_seq[(p, stage)])
            if rc:
                raise A.AfdError(rc, "afd_unpack_split")
        return self.out

    # -- grouped form: the Attention side routes ---------------------------------
    def prepare_grouped(self, seed=0):
        """Draw the Attention side's routing (distinct top-k experts per token,
        seeded) and build each peer's routed rows grouped by expert (stable
        sort of the flattened ids) and its group list, on the device."""
        import torch
        w = self.w
        rng = np.random.default_rng(seed)
        self.g_rows, self.g_list, self.g_n = [], [], []
        for p, n in enumerate(w.seq_lens):
            ids = np.argsort(rng.random((n, w.num_experts)), axis=1)[:, :w.topk]
            order = np.argsort(ids.reshape(-1), kind="stable")
            rows = np.ascontiguousarray(self.host["x"][p][order // w.topk])
            self.g_rows.append(act_tensor(rows, w.act, self.device) if rows.shape[0] else None)
            self.g_list.append(np.bincount(ids.reshape(-1), minlength=w.num_experts))
            self.g_n.append(int(rows.shape[0]))
        dt = torch.bfloat16 if w.act == "bf16" else torch.float32
        self.g_y = [torch.empty((max(r, 1), w.hidden), dtype=dt, device=self.device) for r in self.g_n]

    def pack_grouped_all(self, layer=0, stage=0, with_shared=None):
        ws = (self.w.shared_inter > 0) if with_shared is None else with_shared
        for p, n in enumerate(self.w.seq_lens):
            self.seq += 1
            rows = self.g_rows[p]
            rc = A.afd_pack_grouped(self.ctx, p, stage, layer, rows.data_ptr() if rows is not None else 0,
                                    self.g_n[p], self.g_list[p], self.x[p].data_ptr() if n else 0, n,
                                    ws, self.seq)
            if rc:
                raise A.AfdError(rc, "afd_pack_grouped")
            self.last_seq[(p, stage)] = self.seq

    def forward_grouped(self, layer=0, stage=0):
        slots = list(range(self.w.num_peers))
        return A.afd_ffn_forward_grouped(self.ctx, layer, stage, self.g_n, list(self.w.seq_lens), slots)

    def unpack_grouped_all(self, stage=0, with_shared=None):
        ws = (self.w.shared_inter > 0) if with_shared is None else with_shared
        for p, n in enumerate(self.w.seq_lens):
            rc = A.afd_unpack_grouped(self.ctx, p, stage, self.g_y[p].data_ptr() if self.g_n[p] else 0,
                                      self.g_n[p], self.out[p].data_ptr() if (ws and n) else 0, n,
                                      self.last_seq[(p, stage)])
            if rc:
                raise A.AfdError(rc, "afd_unpack_grouped")
        return self.g_y, self.out

    def poll(self):
        return A.afd_poll_status(self.ctx)

    # -- inspection -----------------------------------------------------------------
    def window(self, direction):
        ptr, n = A.afd_get_window(self.ctx, direction)
        return device_view(ptr, n)

    def workspace(self, which, nbytes=None):
        ptr, cap = A.afd_get_workspace(self.ctx, which)
        return device_view(ptr, cap if nbytes is None else nbytes)

    def weights_numpy(self, layer):
        d = W.weights_to_numpy(self.weights[layer])
        d["Wg"] = self.host["Wg"]
        d["bias"] = self.host["bias"]
        return d

    def close(self):
        if self.ctx:
            A.afd_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class RankSet:
    """Token-level dispatch on one GPU: ffn_size FFN-rank contexts, each with
    its block of the experts (a view into the layer's expert weights, no
    copy) and the shared expert, and one Attention-peer object per peer that
    sends to all of them; flags: AFD_CFG_* of the contexts.  The Attention side's gate is the library's router
    (afd_route_noalloc) on each peer's tokens.  Torch plumbing only."""

    def __init__(self, w: W.Workload, ffn_size, ring_depth=1, gemm=A.AFD_GEMM_TENSOR, layers=None,
                 multiplier=2.0, wait_timeout_ns=0, max_total_tokens=0, device="cuda", flags=0):
        import torch
        self.w, self.F, self.device = w, ffn_size, device
        self.layers = w.layers if layers is None else layers
        self.stream = torch.cuda.current_stream()
        self.host = W.host_inputs(w)
        self.x = [act_tensor(a, w.act, device) for a in self.host["x"]]
        self.Wg = torch.from_numpy(self.host["Wg"]).to(device)
        self.bias = None if self.host["bias"] is None else torch.from_numpy(self.host["bias"]).to(device)
        self.weights = [W.expert_weights(w, layer, device) for layer in range(self.layers)]
        self.ranks, self.experts, self.cfgs = [], [], []
        for r in range(ffn_size):
            first, cnt = A.afd_expert_range(w.num_experts, ffn_size, r)
            cfg = A.make_config(w.num_peers, w.token_cap, w.hidden, cnt, w.topk, w.inter,
                                w.shared_inter, act=w.act, renorm=w.renorm,
                                routed_scaling=w.routed_scaling, ring_depth=ring_depth,
                                max_total_tokens=max_total_tokens or w.total_tokens,
                                max_layers=self.layers, gemm=gemm,
                                routed_cap_multiplier=multiplier,
                                wait_timeout_ns=wait_timeout_ns, flags=flags, ffn_rank=r, ffn_size=ffn_size)
            ctx = A.afd_create(cfg, self.stream.cuda_stream)
            for layer, wt in enumerate(self.weights):
                W13, Wd = wt["W13"], wt["Wd"]
                A.afd_set_layer(ctx, layer, 0, 0, W13[first].data_ptr(), Wd[first].data_ptr(),
                                wt["W13s"].data_ptr() if wt["W13s"] is not None else 0,
                                wt["Wds"].data_ptr() if wt["Wds"] is not None else 0)
            self.ranks.append(ctx)
            self.experts.append((first, cnt))
            self.cfgs.append(cfg)
        self.attn = [A.afd_attn_create(self.ranks, p, w.num_experts, self.stream.cuda_stream)
                     for p in range(w.num_peers)]
        dt = torch.bfloat16 if w.act == "bf16" else torch.float32
        self.out = [torch.empty((max(n, 1), w.hidden), dtype=dt, device=device) for n in w.seq_lens]
        self.ids = [torch.zeros((max(n, 1), w.topk), dtype=torch.int32, device=device)
                    for n in w.seq_lens]
        self.wts = [torch.zeros((max(n, 1), w.topk), dtype=torch.float32, device=device)
                    for n in w.seq_lens]
        self.seq = 0
        self.last_seq = {}

    def route(self):
        """The Attention side's gate on every peer's tokens."""
        w = self.w
        for p, n in enumerate(w.seq_lens):
            if not n:
                continue
            rc = A.afd_route_noalloc(self.x[p].data_ptr(), n, w.hidden,
                                     A.AFD_DTYPE_BF16 if w.act == "bf16" else A.AFD_DTYPE_F32,
                                     self.Wg.data_ptr(),
                                     self.bias.data_ptr() if self.bias is not None else 0,
                                     w.num_experts, w.topk, w.renorm, w.routed_scaling,
                                     self.ids[p].data_ptr(), self.wts[p].data_ptr(),
                                     self.stream.cuda_stream)
            if rc:
                raise A.AfdError(rc, "afd_route_noalloc")

    def dispatch_all(self, stage=0, layer=0, with_shared=None):
        ws = (self.w.shared_inter > 0) if with_shared is None else with_shared
        for p, n in enumerate(self.w.seq_lens):
            self.seq += 1
            rc = A.afd_attn_dispatch(self.attn[p], stage, layer, self.x[p].data_ptr() if n else 0,
                                     n, self.ids[p].data_ptr() if n else 0, ws, self.seq)
            if rc:
                raise A.AfdError(rc, "afd_attn_dispatch")
            self.last_seq[(p, stage)] = self.seq

    def serve_all(self, n_items=1, ranks=None):
        slots = list(range(self.w.num_peers))
        for r in (range(self.F) if ranks is None else ranks):
            rc = A.afd_ffn_serve(self.ranks[r], slots, n_items, A.AFD_FORM_GROUPED)
            if rc:
                raise A.AfdError(rc, "afd_ffn_serve")

    def combine_all(self, stage=0):
        for p, n in enumerate(self.w.seq_lens):
            rc = A.afd_attn_combine(self.attn[p], stage, self.wts[p].data_ptr() if n else 0,
                                    self.out[p].data_ptr() if n else 0, n,
                                    self.last_seq[(p, stage)])
            if rc:
                raise A.AfdError(rc, "afd_attn_combine")
        return self.out

    def poll(self):
        """(first status of the ranks, of the peers)"""
        fr = next((s for s in (A.afd_poll_status(c) for c in self.ranks) if s), 0)
        fa = next((s for s in (A.afd_attn_poll_status(a) for a in self.attn) if s), 0)
        return fr, fa

    def window(self, r, direction):
        ptr, n = A.afd_get_window(self.ranks[r], direction)
        return device_view(ptr, n)

    def rank_weights_numpy(self, r, layer=0):
        first, cnt = self.experts[r]
        d = W.weights_to_numpy(self.weights[layer])
        d["W13"] = np.ascontiguousarray(d["W13"][first:first + cnt])
        d["Wd"] = np.ascontiguousarray(d["Wd"][first:first + cnt])
        d["Wg"] = None
        d["bias"] = None
        return d

    def close(self):
        for a in self.attn:
            A.afd_attn_destroy(a)
        self.attn = []
        for c in self.ranks:
            A.afd_destroy(c)
        self.ranks = []


# ---- routing choice and MXFP4 on torch tensors ----------------------------------
# These calls are short: at decode sizes the host's own work is most of their
# time, so the checks are few and plain, and the library's functions, the
# current stream's handle and the scratch come without intermediate layers.
class _Host:
    """torch, the dtypes' codes, the library's functions: looked up once."""

    def __init__(self):
        import torch
        self.empty = torch.empty
        self.int32, self.uint8, self.f32, self.bf16 = torch.int32, torch.uint8, torch.float32, torch.bfloat16
        self.code = {torch.bfloat16: A.AFD_DTYPE_BF16, torch.float32: A.AFD_DTYPE_F32}
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.raw_stream = raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)
        L = A.lib()
        self.select, self.quantize, self.dequantize = L.afd_route_select, L.afd_mx4_quantize, L.afd_mx4_dequantize
        self.gemm, self.gemm_workspace = L.afd_mx4_gemm, L.afd_mx4_gemm_workspace
        self.ffn, self.ffn_workspace = L.afd_mx4_ffn, L.afd_mx4_ffn_workspace


_host = None


def _get():
    global _host
    if _host is None:
        _host = _Host()
    return _host


def _bad(what):
    raise A.AfdError(A.AFD_ERR_ARG, what)


def _not_cuda():
    raise A.AfdError(A.AFD_ERR_NOT_DEVICE, "a CUDA tensor is wanted")


def _rows_int32(h, t, n, what):
    if t.dtype is not h.int32 or t.dim() != 1 or not t.is_contiguous() or (n >= 0 and t.shape[0] != n):
        _bad(f"{what}: contiguous int32 vector" + (f" of {n} wanted" if n >= 0 else " wanted"))


_INT, _DIM = 2 ** 31 - 1, 65536  # the library's ints; its largest row
_SCORES = {"softmax": A.AFD_SCORE_SOFTMAX, "sigmoid": A.AFD_SCORE_SIGMOID}
_RULES = {"floor": A.AFD_MX4_SCALE_FLOOR, "ceil": A.AFD_MX4_SCALE_CEIL}


def route_select(logits, topk, bias=None, score="softmax", n_groups=1, topk_groups=1, group_top=1,
                 renorm=False, routed_scaling=1.0):
    """afd_route_select of logits [T, E] (bf16 or fp32, any row pitch; on the
    current device): (ids int32 [T, topk], weights fp32 [T, topk])."""
    h = _host or _get()
    code, kind = h.code.get(logits.dtype), _SCORES.get(score)
    if code is None or kind is None or logits.dim() != 2:
        _bad("logits: bf16 or fp32 rows [T, E] wanted, score softmax or sigmoid")
    T, E = logits.shape
    # (the binding passes ints and would wrap larger values)
    if not (T <= _INT and E <= 256 and 0 < topk <= 16 and 0 < n_groups <= 32 and 0 < topk_groups <= 32
            and 0 < group_top <= 2):
        _bad("route_select: sizes out of range")
    ld, step = logits.stride()
    if step != 1 and E > 1:
        _bad("logits: rows of neighbouring elements wanted")
    bias_ptr = 0
    if bias is not None:
        if bias.dtype is not h.f32 or bias.shape != (E,) or not bias.is_contiguous():
            _bad("bias: contiguous fp32 [E] wanted")
        bias_ptr = bias.data_ptr()
    if not logits.is_cuda:
        _not_cuda()
    dev = logits.device
    ids = h.empty((T, topk), dtype=h.int32, device=dev)
    weights = h.empty((T, topk), dtype=h.f32, device=dev)
    rc = h.select(logits.data_ptr(), ld if T > 1 else E, T, code, bias_ptr, E, topk, kind, n_groups, topk_groups,
                  group_top, 1 if renorm else 0, routed_scaling, ids.data_ptr(), weights.data_ptr(),
                  h.raw_stream(dev.index))
    if rc:
        raise A.AfdError(rc, "afd_route_select")
    return ids, weights


class Mx4:
    """MXFP4 rows: codes uint8 [rows, cols / 2], scales uint8 [rows, cols / 32]."""
    __slots__ = ("codes", "scales", "rows", "cols")

    def __init__(self, codes, scales):
        h = _host or _get()
        rows, half = codes.shape if codes.dim() == 2 else _bad("codes: [rows, cols / 2] wanted")
        if (codes.dtype is not h.uint8 or scales.dtype is not h.uint8 or half % 16 or half > _DIM // 2
                or scales.shape != (rows, half // 16) or not codes.is_contiguous() or not scales.is_contiguous()):
            _bad("MXFP4: contiguous uint8 codes [rows, cols / 2] and scales [rows, cols / 32] wanted")
        self.codes, self.scales, self.rows, self.cols = codes, scales, rows, 2 * half


def mx4_quantize(x, src_rows=None, topk=1, rule="floor"):
    """afd_mx4_quantize of x [rows, cols] (bf16 or fp32, any 16-byte row
    pitch); src_rows int32 [n]: row r codes x[src_rows[r] // topk]."""
    h = _host or _get()
    code = h.code.get(x.dtype)
    if code is None or x.dim() != 2 or rule not in _RULES:
        _bad("x: bf16 or fp32 rows wanted, rule floor or ceil")
    n_x, cols = x.shape
    ld, step = x.stride()
    if cols % 32 or cols > _DIM or step != 1 or not 0 < topk <= _INT:
        _bad("x: rows of 32 m neighbouring elements, up to 65536, and topk over 0 wanted")
    n, src = n_x, 0
    if src_rows is not None:
        _rows_int32(h, src_rows, -1, "src_rows")
        n, src = src_rows.shape[0], src_rows.data_ptr()
    if not x.is_cuda:
        _not_cuda()
    dev = x.device
    q = Mx4.__new__(Mx4)
    q.codes = codes = h.empty((n, cols // 2), dtype=h.uint8, device=dev)
    q.scales = scales = h.empty((n, cols // 32), dtype=h.uint8, device=dev)
    q.rows, q.cols = n, cols
    rc = h.quantize(x.data_ptr(), ld if n_x > 1 else cols, n_x, cols, code, src, topk, n, _RULES[rule],
                    codes.data_ptr(), scales.data_ptr(), h.raw_stream(dev.index))
    if rc:
        raise A.AfdError(rc, "afd_mx4_quantize")
    return q


def mx4_dequantize(q, dtype):
    """The values of q as a tensor [rows, cols] of dtype (bf16 or fp32)."""
    h = _host or _get()
    code = h.code.get(dtype)
    if code is None:
        _bad(f"dtype {dtype}: bfloat16 or float32 wanted")
    if not q.codes.is_cuda:
        _not_cuda()
    dev = q.codes.device
    out = h.empty((q.rows, q.cols), dtype=dtype, device=dev)
    rc = h.dequantize(q.codes.data_ptr(), q.scales.data_ptr(), q.rows, q.cols, code, out.data_ptr(), q.cols,
                      h.raw_stream(dev.index))
    if rc:
        raise A.AfdError(rc, "afd_mx4_dequantize")
    return out


class Mx4Weight:
    """Expert weights [E, M, K] in MXFP4 (codes uint8 [E, M, K / 2], scales
    uint8 [E, M, K / 32]) packed for the product; the inputs are not kept."""

    def __init__(self, codes, scales, swiglu=False):
        h = _host or _get()
        if (codes.dim() != 3 or codes.dtype is not h.uint8 or scales.dtype is not h.uint8
                or not codes.is_contiguous() or not scales.is_contiguous()
                or scales.shape != (*codes.shape[:2], codes.shape[2] // 16)):
            _bad("weight: contiguous uint8 codes [E, M, K / 2] and scales [E, M, K / 32] wanted")
        self.experts, self.M, self.K = codes.shape[0], codes.shape[1], 2 * codes.shape[2]
        if self.experts > 256 or self.M > _DIM or self.K > _DIM:
            _bad(f"weight dimensions {(self.experts, self.M, self.K)}")
        self.swiglu = bool(swiglu)
        nbytes = A.afd_mx4_weight_bytes(self.experts, self.M, self.K, self.swiglu)
        if nbytes <= 0:
            _bad(f"weight dimensions {(self.experts, self.M, self.K)}")
        if not codes.is_cuda:
            _not_cuda()
        dev = codes.device
        self.packed = h.empty(nbytes, dtype=h.uint8, device=dev)
        A._check(A.afd_mx4_pack_weight(codes.data_ptr(), scales.data_ptr(), self.experts, self.M, self.K,
                                       self.swiglu, self.packed.data_ptr(), nbytes, h.raw_stream(dev.index)),
                 "afd_mx4_pack_weight")


def _output(h, x, cols, out_dtype, out, dev):
    """(out, its row pitch, the dtype's code)"""
    if out is None:
        out_dtype = h.bf16 if out_dtype is None else out_dtype
        code = h.code.get(out_dtype)
        if code is None:
            _bad(f"out_dtype {out_dtype}: bfloat16 or float32 wanted")
        return h.empty((x.rows, cols), dtype=out_dtype, device=dev), cols, code
    code = h.code.get(out.dtype)
    if code is None or out.shape != (x.rows, cols) or out.stride(1) != 1 or out_dtype not in (None, out.dtype):
        _bad("out: bf16 or fp32 [rows, columns] wanted")
    return out, out.stride(0) if x.rows > 1 else cols, code


def _scratch(h, workspace, need, dev):
    """(pointer, bytes, what keeps it alive until the call is enqueued)"""
    if workspace is not None:
        if not workspace.is_contiguous():
            _bad("workspace: a contiguous tensor wanted")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if need <= 0:
        return 0, 0, None
    t = h.empty(need, dtype=h.uint8, device=dev)
    return t.data_ptr(), need, t


def mx4_gemm(x, offsets, weight, out_dtype=None, out=None, workspace=None):
    """afd_mx4_gemm of the rows x (Mx4) grouped by offsets int32 [E + 1] with
    weight (Mx4Weight): [rows, M], or [rows, M / 2] = silu(gate) * up for a
    swiglu weight.  Rows in no group are not written (out: the caller's)."""
    h = _host or _get()
    _rows_int32(h, offsets, weight.experts + 1, "offsets")
    if x.cols != weight.K:
        _bad(f"rows of {x.cols} columns, weight of {weight.K}")
    if not x.codes.is_cuda:
        _not_cuda()
    dev = x.codes.device
    out, ldo, code = _output(h, x, weight.M // 2 if weight.swiglu else weight.M, out_dtype, out, dev)
    ws, ws_bytes, keep = _scratch(h, workspace, h.gemm_workspace(x.rows, weight.experts, weight.K), dev)
    rc = h.gemm(x.codes.data_ptr(), x.scales.data_ptr(), x.rows, offsets.data_ptr(), weight.experts,
                weight.packed.data_ptr(), weight.M, weight.K, 1 if weight.swiglu else 0, code, out.data_ptr(), ldo,
                ws, ws_bytes, h.raw_stream(dev.index))
    if rc:
        raise A.AfdError(rc, "afd_mx4_gemm")
    return out


def mx4_ffn(x, offsets, w13, wd, out_dtype=None, out=None, workspace=None):
    """afd_mx4_ffn: the expert FFN of the grouped rows x (Mx4) with w13 (a
    swiglu Mx4Weight [E, 2 inter, hidden]) and wd ([E, hidden, inter])."""
    h = _host or _get()
    hidden, inter = wd.M, wd.K
    if (not w13.swiglu or wd.swiglu or w13.experts != wd.experts or w13.K != hidden or w13.M != 2 * inter
            or x.cols != hidden):
        _bad("w13 / wd / x dimensions do not match")
    _rows_int32(h, offsets, wd.experts + 1, "offsets")
    if not x.codes.is_cuda:
        _not_cuda()
    dev = x.codes.device
    out, ldo, code = _output(h, x, hidden, out_dtype, out, dev)
    ws, ws_bytes, keep = _scratch(h, workspace, h.ffn_workspace(x.rows, wd.experts, hidden, inter), dev)
    rc = h.ffn(x.codes.data_ptr(), x.scales.data_ptr(), x.rows, offsets.data_ptr(), wd.experts,
               w13.packed.data_ptr(), wd.packed.data_ptr(), hidden, inter, code, out.data_ptr(), ldo,
               ws, ws_bytes, h.raw_stream(dev.index))
    if rc:
        raise A.AfdError(rc, "afd_mx4_ffn")
    return out
