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
    sends to all of them.  The Attention side's gate is the library's router
    (afd_route_noalloc) on each peer's tokens.  Torch plumbing only."""

    def __init__(self, w: W.Workload, ffn_size, ring_depth=1, gemm=A.AFD_GEMM_TENSOR, layers=None,
                 multiplier=2.0, wait_timeout_ns=0, max_total_tokens=0, device="cuda"):
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
                                wait_timeout_ns=wait_timeout_ns, ffn_rank=r, ffn_size=ffn_size)
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
def _act_code(dtype):
    import torch
    if dtype is torch.bfloat16:
        return A.AFD_DTYPE_BF16
    if dtype is torch.float32:
        return A.AFD_DTYPE_F32
    raise A.AfdError(A.AFD_ERR_ARG, f"dtype {dtype}: bfloat16 or float32 wanted")


def _stream(t):
    """The current stream of t's device; t must live on the current device
    (the library launches there)."""
    import torch
    if t.device.type != "cuda":
        raise A.AfdError(A.AFD_ERR_NOT_DEVICE, "a CUDA tensor is wanted")
    return torch.cuda.current_stream(t.device).cuda_stream


def _want(ok, what):
    if not ok:
        raise A.AfdError(A.AFD_ERR_ARG, what)


def _int32_vector(t, what):
    import torch
    _want(t.dtype is torch.int32 and t.dim() == 1 and t.is_contiguous(), f"{what}: int32 vector wanted")
    return t


def route_select(logits, topk, bias=None, score="softmax", n_groups=1, topk_groups=1, group_top=1,
                 renorm=False, routed_scaling=1.0):
    """afd_route_select of logits [T, E] (bf16 or fp32, any row pitch):
    (ids int32 [T, topk], weights fp32 [T, topk])."""
    import torch
    _want(logits.dim() == 2 and (logits.stride(1) == 1 or logits.shape[1] == 1), "logits: rows [T, E] wanted")
    T, E = logits.shape
    if bias is not None:
        _want(bias.dtype is torch.float32 and bias.shape == (E,) and bias.is_contiguous(),
              "bias: fp32 [E] wanted")
    _want(score in ("softmax", "sigmoid"), f"score {score!r}")
    ids = torch.empty((T, topk), dtype=torch.int32, device=logits.device)
    weights = torch.empty((T, topk), dtype=torch.float32, device=logits.device)
    A._check(A.afd_route_select(logits.data_ptr(), logits.stride(0) if T > 1 else E, T, _act_code(logits.dtype),
                                0 if bias is None else bias.data_ptr(), E, topk,
                                A.AFD_SCORE_SIGMOID if score == "sigmoid" else A.AFD_SCORE_SOFTMAX,
                                n_groups, topk_groups, group_top, renorm, routed_scaling,
                                ids.data_ptr(), weights.data_ptr(), _stream(logits)),
             "afd_route_select")
    return ids, weights


class Mx4:
    """MXFP4 rows: codes uint8 [rows, cols / 2], scales uint8 [rows, cols / 32]."""

    def __init__(self, codes, scales):
        import torch
        _want(codes.dtype is torch.uint8 and scales.dtype is torch.uint8 and codes.dim() == 2
              and codes.is_contiguous() and scales.is_contiguous()
              and codes.shape[1] % 16 == 0 and scales.shape == (codes.shape[0], codes.shape[1] // 16),
              "MXFP4: contiguous uint8 codes [rows, cols / 2] and scales [rows, cols / 32] wanted")
        self.codes, self.scales = codes, scales
        self.rows, self.cols = codes.shape[0], 2 * codes.shape[1]


def mx4_quantize(x, src_rows=None, topk=1, rule="floor"):
    """afd_mx4_quantize of x [rows, cols] (bf16 or fp32, any 16-byte row
    pitch); src_rows int32 [n]: row r codes x[src_rows[r] // topk]."""
    import torch
    _want(x.dim() == 2 and x.shape[1] % 32 == 0 and x.stride(1) == 1, "x: rows [n, 32 m] wanted")
    _want(rule in ("floor", "ceil"), f"rule {rule!r}")
    n = x.shape[0] if src_rows is None else _int32_vector(src_rows, "src_rows").numel()
    q = Mx4(torch.empty((n, x.shape[1] // 2), dtype=torch.uint8, device=x.device),
            torch.empty((n, x.shape[1] // 32), dtype=torch.uint8, device=x.device))
    A._check(A.afd_mx4_quantize(x.data_ptr(), x.stride(0) if x.shape[0] > 1 else x.shape[1], x.shape[0],
                                x.shape[1], _act_code(x.dtype),
                                0 if src_rows is None else src_rows.data_ptr(), topk, n,
                                A.AFD_MX4_SCALE_CEIL if rule == "ceil" else A.AFD_MX4_SCALE_FLOOR,
                                q.codes.data_ptr(), q.scales.data_ptr(), _stream(x)),
             "afd_mx4_quantize")
    return q


def mx4_dequantize(q, dtype):
    """The values of q as a tensor [rows, cols] of dtype (bf16 or fp32)."""
    import torch
    out = torch.empty((q.rows, q.cols), dtype=dtype, device=q.codes.device)
    A._check(A.afd_mx4_dequantize(q.codes.data_ptr(), q.scales.data_ptr(), q.rows, q.cols,
                                  _act_code(dtype), out.data_ptr(), q.cols, _stream(q.codes)),
             "afd_mx4_dequantize")
    return out


class Mx4Weight:
    """Expert weights [E, M, K] in MXFP4 (codes uint8 [E, M, K / 2], scales
    uint8 [E, M, K / 32]) packed for the product; the inputs are not kept."""

    def __init__(self, codes, scales, swiglu=False):
        import torch
        _want(codes.dim() == 3 and codes.dtype is torch.uint8 and scales.dtype is torch.uint8
              and codes.is_contiguous() and scales.is_contiguous()
              and scales.shape == (*codes.shape[:2], codes.shape[2] // 16),
              "weight: contiguous uint8 codes [E, M, K / 2] and scales [E, M, K / 32] wanted")
        self.experts, self.M, self.K = codes.shape[0], codes.shape[1], 2 * codes.shape[2]
        self.swiglu = bool(swiglu)
        nbytes = A.afd_mx4_weight_bytes(self.experts, self.M, self.K, self.swiglu)
        _want(nbytes > 0, f"weight dimensions {(self.experts, self.M, self.K)}")
        self.packed = torch.empty(nbytes, dtype=torch.uint8, device=codes.device)
        A._check(A.afd_mx4_pack_weight(codes.data_ptr(), scales.data_ptr(), self.experts, self.M, self.K,
                                       self.swiglu, self.packed.data_ptr(), nbytes, _stream(codes)),
                 "afd_mx4_pack_weight")


def mx4_gemm(x, offsets, weight, out_dtype=None, out=None):
    """afd_mx4_gemm of the rows x (Mx4) grouped by offsets int32 [E + 1] with
    weight (Mx4Weight): [rows, M], or [rows, M / 2] = silu(gate) * up for a
    swiglu weight.  Rows in no group are not written (out: the caller's)."""
    import torch
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    _want(_int32_vector(offsets, "offsets").numel() == weight.experts + 1, "offsets: int32 [E + 1] wanted")
    _want(x.cols == weight.K, f"rows of {x.cols} columns, weight of {weight.K}")
    cols = weight.M // 2 if weight.swiglu else weight.M
    if out is None:
        out = torch.empty((x.rows, cols), dtype=out_dtype, device=x.codes.device)
    _want(out.shape == (x.rows, cols) and out.stride(1) == 1 and out.dtype is out_dtype, "out")
    A._check(A.afd_mx4_gemm(x.codes.data_ptr(), x.scales.data_ptr(), x.rows, offsets.data_ptr(),
                            weight.experts, weight.packed.data_ptr(), weight.M, weight.K, weight.swiglu,
                            _act_code(out_dtype), out.data_ptr(), out.stride(0) if x.rows > 1 else cols,
                            _stream(x.codes)),
             "afd_mx4_gemm")
    return out


def mx4_ffn(x, offsets, w13, wd, out_dtype=None, out=None, workspace=None):
    """afd_mx4_ffn: the expert FFN of the grouped rows x (Mx4) with w13 (a
    swiglu Mx4Weight [E, 2 inter, hidden]) and wd ([E, hidden, inter])."""
    import torch
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    hidden, inter = wd.M, wd.K
    _want(w13.swiglu and not wd.swiglu and w13.experts == wd.experts and w13.K == hidden
          and w13.M == 2 * inter and x.cols == hidden, "w13 / wd / x dimensions do not match")
    _want(_int32_vector(offsets, "offsets").numel() == wd.experts + 1, "offsets: int32 [E + 1] wanted")
    if out is None:
        out = torch.empty((x.rows, hidden), dtype=out_dtype, device=x.codes.device)
    _want(out.shape == (x.rows, hidden) and out.stride(1) == 1 and out.dtype is out_dtype, "out")
    if workspace is None:
        workspace = torch.empty(max(A.afd_mx4_ffn_workspace(x.rows, inter), 1), dtype=torch.uint8,
                                device=x.codes.device)
    A._check(A.afd_mx4_ffn(x.codes.data_ptr(), x.scales.data_ptr(), x.rows, offsets.data_ptr(), wd.experts,
                           w13.packed.data_ptr(), wd.packed.data_ptr(), hidden, inter,
                           _act_code(out_dtype), out.data_ptr(), out.stride(0) if x.rows > 1 else hidden,
                           workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                           _stream(x.codes)),
             "afd_mx4_ffn")
    return out
