"""Chains the library's calls for one expert layer over preallocated buffers:
route statistics -> plan -> forward (-> backward plan -> backward).

Buffers come from torch (device memory); every computation is a library call.
"""
from __future__ import annotations

import torch

from . import binding as B


class LayerRunner:
    def __init__(self, w1, w2, w1_scale=None, w2_scale=None, *, act_dtype, T, k, beta, P, s,
                 owner, lam=12, with_backward=False, save_z=None, quota_umin=None,
                 gate_rho=None, two_phase=False):
        dev = w1.device
        self.dev = dev
        self.layer = B.make_layer(w1, w2, w1_scale, w2_scale, act_dtype)
        self.keep = (w1, w2, w1_scale, w2_scale)
        self.E, self.d, self.dff = self.layer.E, self.layer.d, self.layer.d_ff
        self.T, self.k, self.beta, self.P, self.s, self.lam = T, k, beta, P, s, lam
        # quota_umin set: every plan (forward and backward) comes from the
        # quota-driven solver with that quota floor
        self.quota_umin = quota_umin
        # gate_rho set: every plan passes the replication gate with that price
        # per replica (thousandths of a block)
        self.gate_rho = gate_rho
        self.act_dtype = act_dtype
        # two_phase: FC1 / FC2 (dA / dX) in one two-phase launch instead of two
        self.two_phase = two_phase
        # producer workgroups per worker of the forward / backward two-phase
        # launch (0: every workgroup runs both phases)
        self.split_fwd = 0
        self.split_bwd = 0
        # e4m3 weights: every product but the weight gradients on the fp8 MFMA
        # (x, A, dy and dZ quantized per row block of 128 features)
        self.fp8_act = False
        self.owner = owner.to(device=dev, dtype=torch.int32).contiguous()
        self.with_backward = with_backward
        self.ws = B.workspace(self.layer, T, k, beta, P, s, with_backward, dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.rs = B.alloc_route(T, k, self.E, beta, dev)
        nbc = B.max_blocks(T, k, self.E, beta)
        self.plan_f = B.alloc_plan(self.E, P, nbc, dev)
        self.plan_b = B.alloc_plan(self.E, P, nbc, dev) if with_backward else None
        # the backward plan needs only the routing statistics: it runs on this
        # stream (default priority) while the forward plan and the forward run
        self.side = torch.cuda.Stream(device=dev) if with_backward and dev.type == "cuda" else None
        self.y = torch.empty((T, self.d), dtype=act_dtype, device=dev)
        need_z = with_backward if save_z is None else save_z
        ms = max(B.max_slots(T, k, self.E, beta), 1)
        self.z = torch.empty((ms, 2 * self.dff), dtype=act_dtype, device=dev) if need_z else None
        if with_backward:
            self.dx = torch.empty((T, self.d), dtype=act_dtype, device=dev)
            self.dw1 = torch.empty((self.E, 2 * self.dff, self.d), dtype=torch.float32, device=dev)
            self.dw2 = torch.empty((self.E, self.d, self.dff), dtype=torch.float32, device=dev)

    def route(self, topk_ids):
        return B.route_stats(topk_ids, self.E, self.beta, self.rs, self.ws, self.status)

    def make_plan(self, mode=B.PLAN_FWD, s=None, out=None):
        if s is not None and s > self.s:
            raise B.MoeError(f"replica budget s={s} above the runner's s={self.s}")
        out = self.plan_f if out is None else out
        lam = self.lam
        if self.quota_umin is not None:
            mode, lam = B.PLAN_QUOTA, self.quota_umin
        B.plan(self.rs["block_counts"], self.rs["block_offsets"], self.owner, self.P,
               self.s if s is None else s, mode, lam, out, self.ws, self.status)
        if self.gate_rho is not None:
            B.plan_gate(self.rs["block_counts"], self.rs["block_offsets"], self.owner, self.P,
                        self.gate_rho, out, self.status)
        return out

    def forward(self, x, gates, topk_ids, block_worker=None, events=None, timeline=None):
        bw = self.plan_f["block_worker"] if block_worker is None else block_worker
        B.forward(self.layer, x, gates, topk_ids, self.beta, self.P, self.rs, bw, self.y, self.z,
                  self.ws, self.status, events, timeline, self.two_phase, self.split_fwd,
                  self.fp8_act)
        return self.y

    def backward(self, x, gates, dy, topk_ids, block_worker=None, events=None, timeline=None,
                 dlogp=None):
        """dx, dw1, dw2; into dlogp [T][k] (optional) the gates' gradients in log form, p dL/dp."""
        bw = self.plan_b["block_worker"] if block_worker is None else block_worker
        B.backward(self.layer, x, gates, dy, self.z, topk_ids, self.beta, self.P, self.s, self.rs,
                   self.owner, bw, self.dx, self.dw1, self.dw2, self.ws, self.status, events,
                   timeline, self.two_phase, self.split_bwd, self.fp8_act, dlogp)
        return self.dx, self.dw1, self.dw2

    def step(self, x, gates, topk_ids, dy=None, s=None, timeline=None):
        """One pass of the whole path: route -> plan -> forward [-> plan(bwd) -> backward].

        s (default: the runner's s) is the replica budget of both plans; it may
        not exceed the runner's, whose replica slots the backward provides."""
        if s is not None and s > self.s:
            raise B.MoeError(f"replica budget s={s} above the runner's s={self.s}")
        self.route(topk_ids)
        if dy is not None:
            self.plan_bwd_async(s)
        self.make_plan(B.PLAN_FWD, s)
        self.forward(x, gates, topk_ids, timeline=timeline)
        if dy is not None:
            self.join_bwd_plan()
            self.backward(x, gates, dy, topk_ids, timeline=timeline)
        return self.y

    def plan_bwd_async(self, s=None, events=None):
        """The backward plan on the side stream, after the work already queued
        on the current stream (the routing statistics); `events` (optional,
        a B.Events of 2) brackets it there."""
        main = torch.cuda.current_stream(self.dev)
        self.side.wait_stream(main)
        with torch.cuda.stream(self.side):
            if events is not None:
                events.record(0)
            self.make_plan(B.PLAN_BWD, s, self.plan_b)
            if events is not None:
                events.record(1)

    def join_bwd_plan(self):
        """The current stream waits for the backward plan."""
        torch.cuda.current_stream(self.dev).wait_stream(self.side)


def _share(a, others):
    """Whether tensor a lies in the memory of one of the others (all of them allocations of their own)."""
    at = a.untyped_storage().data_ptr()                  # 0: empty
    return at != 0 and any(t.untyped_storage().data_ptr() == at for t in others)


class BlockRunner(LayerRunner):
    """The expert layer as a block of a model, trained: norm -> router -> layer -> norm, gate and
    residual, its gradients, and AdamW on its weights.

        n = w_in x / rms(x);  logits = n w_router^T;  ids, gates, losses = router(logits)
        out = x + alpha gate (w_out y / rms(y)),  y = layer(n, gates, ids)

    w_router [E][d] and the norms' weights w_in, w_out [d] are of the activation dtype, gate [d] is
    fp32 (None: 1).  The two products with w_router are plain library products; every other step
    is a library call of its own over buffers made here, on the current stream."""

    def __init__(self, w1, w2, w_router, w_in, w_out, gate=None, w1_scale=None, w2_scale=None, *,
                 score="softmax", renorm=True, scale=1.0, alpha=1.0, eps=1e-6, **layer):
        super().__init__(w1, w2, w1_scale, w2_scale, **layer)
        T, d, dev, dt = self.T, self.d, self.dev, self.act_dtype
        if tuple(w_router.shape) != (self.E, d) or w_router.dtype != dt:
            raise B.MoeError(f"w_router: expected {(self.E, d)} of {dt}, got "
                             f"{tuple(w_router.shape)} of {w_router.dtype}")
        if gate is not None and tuple(gate.shape) != (d,):
            raise B.MoeError(f"gate: expected {(d,)}, got {tuple(gate.shape)}")
        self.w_router, self.w_in, self.w_out, self.gate = w_router, w_in, w_out, gate
        self.alpha, self.eps = alpha, eps
        self.router = B.make_router(self.E, self.k, dt, score, renorm, scale)
        self.routed = B.alloc_router(self.router, T, dev)
        self.router_ws = B.router_workspace(self.router, T, dev)
        rows = dict(dtype=dt, device=dev)
        f32 = dict(dtype=torch.float32, device=dev)
        self.n, self.out = torch.empty((T, d), **rows), torch.empty((T, d), **rows)
        self.logits = torch.empty((T, self.E), **rows)
        self.rstd_in, self.rstd_out = torch.empty(T, **f32), torch.empty(T, **f32)
        self.optimizer = self.x = None
        if self.with_backward:
            self.norm_ws = B.norm_workspace(T, d, dev)
            self.dy, self.dn = torch.empty((T, d), **rows), torch.empty((T, d), **rows)
            self.dx_block = torch.empty((T, d), **rows)
            self.dlogits = torch.empty((T, self.E), **rows)
            self.dw_router = torch.empty((self.E, d), **rows)
            self.dlogp = torch.empty((T, self.k), **f32)
            self.dw_in, self.dw_out = torch.empty(d, **f32), torch.empty(d, **f32)
            self.dgate = None if gate is None else torch.empty(d, **f32)

    def block_forward(self, x, mask=None):
        """out [T][d] of x [T][d]; mask [T] (optional): 0 where a row is padding, which, whatever it
        holds, passes the residual alone and reaches no weight's gradient.  The routing's losses are
        in self.routed["losses"].  x may be the out of an earlier call, which this one overwrites: such
        a call has no backward pass, which would read x again."""
        own = [self.n, self.y] + ([self.dy, self.dn, self.dx, self.dx_block] if self.with_backward else [])
        if _share(x, own):
            raise B.MoeError("x lies in a buffer of the runner that the call overwrites")
        self.x, self.mask = None if _share(x, [self.out]) else x, mask
        B.norm_in(x, self.w_in, self.eps, self.n, self.rstd_in, mask=mask)
        torch.mm(self.n, self.w_router.t(), out=self.logits)
        r = B.router_forward(self.router, self.logits, self.routed, self.router_ws, self.status, mask)
        self.route(r["topk_ids"])
        if self.with_backward:
            self.plan_bwd_async()
        self.make_plan()
        self.forward(self.n, r["gates"], r["topk_ids"])
        if self.with_backward:                 # the next call rewrites what the plan reads
            self.join_bwd_plan()
        return B.norm_out(self.y, x, self.w_out, self.eps, self.out, self.rstd_out, self.gate,
                          self.alpha, mask)

    def block_backward(self, dout, dlosses=None):
        """Gradients of block_forward's last call from dout [T][d] and (optional) dlosses [2], those
        of the balance and z losses: dx, and dw1, dw2, dw_router, dw_in, dw_out, dgate in self."""
        if not self.with_backward or self.x is None:
            raise B.MoeError("block_backward needs a runner with a backward pass, after block_forward of an "
                             "x that is not the runner's out")
        if _share(dout, [self.dy, self.dn, self.dx]):
            raise B.MoeError("dout lies in a buffer of the runner that the call overwrites")
        r = self.routed
        B.norm_out_backward(dout, self.y, self.w_out, self.rstd_out, self.dy, self.dw_out,
                            self.norm_ws, self.gate, self.alpha, self.dgate, self.mask)
        self.backward(self.n, r["gates"], self.dy, r["topk_ids"], dlogp=self.dlogp)
        B.router_backward(self.router, self.logits, r, self.dlogp, dlosses, self.dlogits, self.mask)
        torch.mm(self.dlogits.t(), self.n, out=self.dw_router)
        torch.addmm(self.dx, self.dlogits, self.w_router, out=self.dn)
        return B.norm_in_backward(self.dn, self.x, self.w_in, self.rstd_in, self.dx_block, self.dw_in,
                                  self.norm_ws, dr=dout, mask=self.mask)

    def make_optimizer(self, state_bits=32):
        """AdamW states (zeros) for the block's weights; state_bits 32 (fp32) or 8 (e4m3 codes and
        a scale for 128 of them).  One list: all weights, the norms' and the gate too, take the same rate
        and decay, and bf16 ones have no fp32 copy.  Where they shall not, binding.make_adamw takes lists of
        any of these weights and gradients."""
        if not self.with_backward or self.layer.w_dtype == B.MOE_FP8_E4M3:
            raise B.MoeError("the optimizer needs a runner with a backward pass and fp32 or bf16 weights")
        w1, w2 = self.keep[:2]
        p = [w1, w2, self.w_router, self.w_in, self.w_out]
        g = [self.dw1, self.dw2, self.dw_router, self.dw_in, self.dw_out]
        if self.gate is not None:
            p.append(self.gate)
            g.append(self.dgate)
        if state_bits not in (8, 32):
            raise B.MoeError(f"state_bits={state_bits}: 8 or 32")
        dt = torch.uint8 if state_bits == 8 else torch.float32
        states = lambda: [torch.zeros(t.shape, dtype=dt, device=self.dev) for t in p]
        scales = lambda: [torch.zeros(-(-t.numel() // B.ADAMW_BLOCK), device=self.dev) for t in p] \
            if state_bits == 8 else None
        self.state = {"m": states(), "v": states(), "m_scale": scales(), "v_scale": scales()}
        self.optimizer = B.make_adamw(p, g, **self.state)
        return self.optimizer

    def optimizer_step(self, lr, step, **hyper):
        """One AdamW step (binding.adamw's arguments) on the block's weights, in place."""
        if self.optimizer is None:
            raise B.MoeError("make_optimizer first")
        B.adamw(self.optimizer, lr, step=step, **hyper)
