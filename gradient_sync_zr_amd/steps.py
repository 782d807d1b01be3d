"""Host-side drivers of the reduction path: what a data-parallel trainer's
reducer does with the C ABI, one step at a time.

* :class:`Zero2GradSync` - a flat per-rank gradient reduced bucket by bucket
  through the scheduler (ping-pong buffer indices, per-buffer completion
  events), each bucket a fused reduce-scatter + average + cast into the
  rank's fp32 partitioned flat gradient ("ZeRO-1/2 average_tensor serializes
  backward compute behind the preceding reduction", Proposed design
  direction; "DeepSpeed ZeRO-3 源码解析", 3.1 bucketing, 5.3 partition write,
  5.4 epilogue flush).
* :class:`Zero3Gather` - full parameters gathered from 1/K shards in greedy
  prefetch buckets ("DeepSpeed ZeRO-3 源码解析", 2.1 fetch/prefetch and 2.2
  the prefetch size cap), one all-gather launch set per bucket.
* :class:`CkptNormLinear` - one rank's norm and the linear layer behind it,
  whose activations are kept as 8-bit checkpoints and whose backward pass
  writes the weight gradients into the rank's flat gradient, where
  :class:`Zero2GradSync` takes them (its ``produce`` hook is the place to call
  the backward pass from).
* :class:`PackedNormLinear` - the same place in a layer with an RMS norm, whose
  products run on packed activations and packed weights too.
* :class:`ClipAdamW` - the step behind the reduction: the partitions' global
  norm, clipping, AdamW, and the bf16 shards that :class:`Zero3Gather` gathers.

All tensors are torch CUDA tensors used only as device memory; every
computation happens in libzr's kernels.
"""
from __future__ import annotations

from typing import Callable, List, Optional, Sequence

from . import (ZR_BF16, ZR_CKPT_E2M1, ZR_CKPT_E4M3, ZR_FP32, ZR_ORDER_RING, Sched, tensor_table, zr_adamw, zr_all_gather,
               zr_ckpt_bytes, zr_ckpt_format_bytes, zr_ckpt_linear, zr_ckpt_linear_workspace_bytes, zr_ckpt_pack,
               zr_ckpt_pack_t, zr_ckpt_wgrad, zr_ckpt_wgrad_workspace_bytes, zr_grad_norm,
               zr_grad_norm_workspace_bytes, zr_layernorm_bwd, zr_layernorm_fwd, zr_layernorm_workspace_bytes,
               zr_plan_buckets, zr_rmsnorm_bwd, zr_rmsnorm_fwd, zr_rmsnorm_workspace_bytes, _dtype)


def ceil_div(a: int, b: int) -> int:
    return -(-a // b)


class Zero2GradSync:
    """Bucketed reduce-scatter of K flat gradients into K fp32 partitions.

    grads[r]      : rank r's flat gradient, N_total elements (bf16 or fp32)
    partitions[r] : rank r's partitioned flat gradient; bucket b's chunk is
                    written at the sum of the previous buckets' chunk sizes
    bucket        : elements per bucket (the last bucket takes the rest)
    """

    def __init__(self, grads: Sequence, partitions: Sequence, bucket: int, chunk_shift: int = 1,
                 average: bool = True, order: int = ZR_ORDER_RING, n_buffers: int = 2,
                 reduction_stream=None):
        self.K = len(grads)
        self.grads, self.partitions = list(grads), list(partitions)
        self.N_total = grads[0].numel()
        self.in_dt, self.out_dt = _dtype(grads[0]), _dtype(partitions[0])
        self.in_es = 2 if self.in_dt == ZR_BF16 else 4
        self.out_es = 2 if self.out_dt == ZR_BF16 else 4
        self.shift, self.average, self.order = chunk_shift, average, order
        self.n_buffers = n_buffers
        self.buckets = []  # (N_b, input pointers, output pointers)
        start, poff = 0, 0
        while start < self.N_total:
            n = min(bucket, self.N_total - start)
            C = ceil_div(n, self.K)
            ins = [g.data_ptr() + start * self.in_es for g in self.grads]
            outs = [p.data_ptr() + poff * self.out_es for p in self.partitions]
            self.buckets.append((n, ins, outs, start, poff))
            start += n
            poff += C
        self.partition_numel = poff
        for p in self.partitions:
            if p.numel() < poff:
                raise ValueError(f"partition holds {p.numel()} elements, needs {poff}")
        if reduction_stream is None:
            import torch
            reduction_stream = torch.cuda.current_stream()  # what the scheduler then takes
        self.reduction_stream = reduction_stream
        self.sched = Sched(n_buffers=n_buffers, max_producers=1,
                           reduction_stream=reduction_stream)

    def step(self, producer_stream=None, timing: Optional[List] = None,
             micro_step: int = 0, produce: Optional[Callable] = None) -> None:
        """One gradient sync. `produce(i, stream)`, if given, enqueues the work
        that writes bucket i's gradients (the backward pass) on the producer
        stream, after the stream has waited for the buffer to be free and
        before the bucket's reduction, which waits for it. `timing`, if given,
        receives (start, end) torch events recorded on the reduction stream
        around each bucket's launch, after the reduction stream has waited for the
        producer. Micro-step 0 overwrites the partitions;
        later micro-steps of a gradient-accumulation window add to them
        ("DeepSpeed ZeRO-3 源码解析", 5.3 and 6)."""
        import torch
        prod = producer_stream if producer_stream is not None else torch.cuda.current_stream()
        for i, (n, ins, outs, _, _) in enumerate(self.buckets):
            buf = i % self.n_buffers
            self.sched.acquire(buf, prod)
            if produce is not None:
                produce(i, prod)
            if timing is not None:
                e0 = torch.cuda.Event(enable_timing=True)
                e1 = torch.cuda.Event(enable_timing=True)
                # the reduction's wait on the producer comes before the start
                # event, so the pair brackets the launch alone (the launch's
                # own wait then finds the producer's work done)
                self.reduction_stream.wait_stream(prod)
                e0.record(self.reduction_stream)
            self.sched.submit_rs(buf, [prod], ins, n, outs, chunk_shift=self.shift,
                                 average=self.average, order=self.order, in_dtype=self.in_dt,
                                 out_dtype=self.out_dt, accumulate=micro_step > 0)
            if timing is not None:
                e1.record(self.reduction_stream)
                timing.append((e0, e1))
        self.sched.flush(prod)

    def close(self):
        self.sched.close()


class Zero3Gather:
    """Gather K full parameter buffers from K shard buffers, bucket by bucket.

    numels      : parameter sizes in trace order
    cap         : prefetch bucket size in elements
    Shard p of every rank is ceil(numel_p / K) elements at the running offset
    of the shard buffer; parameter p sits at the running offset of the full
    buffer.
    """

    def __init__(self, shards: Sequence, fulls: Sequence, numels: Sequence[int], cap: int,
                 chunk_shift: int = 0):
        self.K = len(shards)
        self.shards, self.fulls = list(shards), list(fulls)
        self.dt = _dtype(shards[0])
        self.shift = chunk_shift
        bucket_of, nb = zr_plan_buckets(list(numels), cap)
        self.buckets: List[List[tuple]] = [[] for _ in range(nb)]
        soff, foff = 0, 0
        self.param_offsets = []
        for p, n in enumerate(numels):
            self.buckets[bucket_of[p]].append((soff, foff, n))
            self.param_offsets.append((soff, foff, n))
            soff += ceil_div(n, self.K)
            foff += n
        self.shard_numel, self.full_numel = soff, foff
        self._sp = [t.data_ptr() for t in self.shards]
        self._fp = [t.data_ptr() for t in self.fulls]

    def step(self, stream=None) -> None:
        for segs in self.buckets:
            zr_all_gather(self._sp, self._fp, segs, chunk_shift=self.shift, dtype=self.dt,
                          stream=stream)


class CkptNormLinear:
    """Layer norm of a rank's activations (rows x cols) and the linear layer
    that reads it (out_cols x cols), with 8-bit checkpoints.

    flat_grad : the rank's flat gradient; the layer's part of it starts at
                element `offset` and holds, in order, the norm's weight and
                bias (cols each), the linear layer's weight (out_cols x cols)
                and, with `bias`, its bias (out_cols): `numel` elements
    recompute : keep the checkpoint of the norm's input alone, and recompute the
                linear layer's input from it in the backward pass; otherwise
                both checkpoints are kept
    scratch   : a uint8 tensor of `scratch_bytes` elements, the backward pass's
                workspace (and with `recompute` its checkpoint of the linear
                layer's input); layers whose backward passes run one after
                another on a stream may share it, others must not

    The matrix products y W^T of the forward pass and dz W of the backward pass
    are the caller's; they come between the methods:
        forward(x, w, b, y);  z = y W^T
        backward_linear(dz);  dy = dz W;  backward_norm(dy, w, dx)

    Statistics: backward_norm takes xh = (held x - mean) * rstd with the mean and
    rstd of the forward pass, of x itself. With `recompute`, backward_linear
    norms the held x anew, with the held values' own mean and rstd; so the y that
    it multiplies differs from the forward pass's, and its xh from
    backward_norm's, by what the 8 bits lost.

    The layer's buffers belong to the stream that is current when it is made: it
    has to outlive what its methods enqueue on another.
    """

    def __init__(self, flat_grad, offset: int, rows: int, cols: int, out_cols: int, scratch=None,
                 format: int = ZR_CKPT_E4M3, eps: float = 1e-5, bias: bool = True, recompute: bool = True):
        import torch
        self.rows, self.cols, self.out_cols = rows, cols, out_cols
        self.format, self.eps, self.recompute = format, eps, recompute
        sizes = [cols, cols, out_cols * cols] + ([out_cols] if bias else [])
        self.numel = sum(sizes)
        if offset < 0 or offset + self.numel > flat_grad.numel():
            raise ValueError(f"the flat gradient holds {flat_grad.numel()} elements, the layer needs {self.numel} "
                             f"at {offset}")
        parts = flat_grad[offset:offset + self.numel].split(sizes)
        self.dw_norm, self.db_norm = parts[0], parts[1]
        self.dw = parts[2].view(out_cols, cols)
        self.db = parts[3] if bias else None
        self._ws_bytes = max(zr_layernorm_workspace_bytes(rows, cols),
                             zr_ckpt_wgrad_workspace_bytes(rows, out_cols, cols))
        nbytes = zr_ckpt_bytes(rows, cols)
        self._y_at = ceil_div(self._ws_bytes, 256) * 256
        self.scratch_bytes = self._y_at + (nbytes if recompute else 0)
        dev = flat_grad.device
        if scratch is None:
            scratch = torch.empty(self.scratch_bytes, dtype=torch.uint8, device=dev)
        if scratch.numel() < self.scratch_bytes:
            raise ValueError(f"scratch holds {scratch.numel()} bytes, needs {self.scratch_bytes}")
        self.scratch = scratch
        self.ckpt_x = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        self.ckpt_y = scratch[self._y_at:self._y_at + nbytes] if recompute else \
            torch.empty(nbytes, dtype=torch.uint8, device=dev)
        self.mean = torch.empty(rows, dtype=torch.float32, device=dev)
        self.rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        self._params = None

    def forward(self, x, weight, bias, y, stream=None) -> None:
        """The norm of x into y; x itself is not needed afterwards."""
        zr_layernorm_fwd(x, self.rows, self.cols, y, weight, bias, eps=self.eps, mean=self.mean, rstd=self.rstd,
                         ckpt_x=self.ckpt_x, ckpt_y=None if self.recompute else self.ckpt_y,
                         ckpt_format=self.format, stream=stream)
        self._params = (weight, bias, y.dtype)

    def backward_linear(self, dz, accumulate: bool = False, stream=None) -> None:
        """The linear layer's gradients from its output's, dz (rows x
        out_cols), into the flat gradient (added to with accumulate: a later
        micro-step)."""
        if self._params is None:
            raise ValueError("backward before forward")
        if self.recompute:
            weight, bias, y_dtype = self._params
            zr_layernorm_fwd(self.ckpt_x, self.rows, self.cols, None, weight, bias, eps=self.eps,
                             ckpt_y=self.ckpt_y, ckpt_format=self.format, x_dtype=self.format, y_dtype=y_dtype,
                             stream=stream)
        zr_ckpt_wgrad(dz, self.ckpt_y, self.rows, self.out_cols, self.cols, self.dw, dbias=self.db,
                      format=self.format, accumulate=accumulate, workspace=self._workspace(), stream=stream)

    def backward_norm(self, dy, weight, dx=None, accumulate: bool = False, add_dx: bool = False,
                      stream=None) -> None:
        """The norm's gradients from its output's, dy: the weight's and the
        bias's into the flat gradient, the input's into dx (added to with
        add_dx: the residual stream's gradient)."""
        if self._params is None:
            raise ValueError("backward before forward")
        zr_layernorm_bwd(dy, self.ckpt_x, self.rows, self.cols, self.mean, self.rstd, weight, dx=dx,
                         dweight=self.dw_norm, dbias=self.db_norm, accumulate=accumulate, add_dx=add_dx,
                         workspace=self._workspace(), x_dtype=self.format, stream=stream)

    def _workspace(self):
        return self.scratch[:self._ws_bytes]


class PackedNormLinear:
    """RMS norm of a rank's residual stream (rows x cols), and the linear layer
    that reads it (out_cols x cols), on packed operands: activations and output
    gradients in e4m3, the weight in `weight_format` (e4m3 or e2m1), packed once
    per update for both directions.

    flat_grad : the rank's flat gradient; the layer's part of it starts at
                element `offset` and holds, in order, the norm's weight (cols),
                the linear layer's weight (out_cols x cols) and, with `bias`, its
                bias (out_cols): `numel` elements
    scratch   : a uint8 tensor of `scratch_bytes` elements, the calls' workspace;
                layers that run one after another on a stream may share it, others
                must not

        pack_weight(W)                                        after every update of W
        forward(x, norm_weight, z, residual=r, h=h, bias=b)   z = norm(x + r) W^T + b
        backward(dz, norm_weight, dx)                         the flat gradient, and dx

    forward takes a bias where the layer was made with `bias` (the default), and only
    there: its gradient's place in the flat gradient is written by every backward pass.

    dx is the gradient of h = x + r, so of x and of the residual; with add_dx it is
    added to what passed by the norm. h is kept as an 8-bit checkpoint: h, x and the
    residual are not needed after the forward pass. dW takes dz as it is, dx takes
    it packed.

    The layer's buffers belong to the stream that is current when it is made: it
    has to outlive what its methods enqueue on another.
    """

    def __init__(self, flat_grad, offset: int, rows: int, cols: int, out_cols: int, scratch=None,
                 weight_format: int = ZR_CKPT_E4M3, eps: float = 1e-5, bias: bool = True):
        import torch
        if weight_format not in (ZR_CKPT_E4M3, ZR_CKPT_E2M1):
            raise ValueError(f"weight_format {weight_format} is not one of the products', e4m3 or e2m1")
        self.rows, self.cols, self.out_cols = rows, cols, out_cols
        self.weight_format, self.eps = weight_format, eps
        sizes = [cols, out_cols * cols] + ([out_cols] if bias else [])
        self.numel = sum(sizes)
        if offset < 0 or offset + self.numel > flat_grad.numel():
            raise ValueError(f"the flat gradient holds {flat_grad.numel()} elements, the layer needs {self.numel} "
                             f"at {offset}")
        parts = flat_grad[offset:offset + self.numel].split(sizes)
        self.dw_norm = parts[0]
        self.dw = parts[1].view(out_cols, cols)
        self.db = parts[2] if bias else None
        self.scratch_bytes = max(1, zr_rmsnorm_workspace_bytes(rows, cols),
                                 zr_ckpt_linear_workspace_bytes(rows, cols, out_cols),
                                 zr_ckpt_linear_workspace_bytes(rows, out_cols, cols),
                                 zr_ckpt_wgrad_workspace_bytes(rows, out_cols, cols))
        dev = flat_grad.device

        def buffer(r, c, fmt):
            return torch.empty(zr_ckpt_format_bytes(r, c, fmt), dtype=torch.uint8, device=dev)

        if scratch is None:
            scratch = torch.empty(self.scratch_bytes, dtype=torch.uint8, device=dev)
        if scratch.numel() < self.scratch_bytes:
            raise ValueError(f"scratch holds {scratch.numel()} bytes, needs {self.scratch_bytes}")
        self.scratch = scratch[:self.scratch_bytes]
        self.w, self.w_t = buffer(out_cols, cols, weight_format), buffer(cols, out_cols, weight_format)
        self.ckpt_h, self.ckpt_y = buffer(rows, cols, ZR_CKPT_E4M3), buffer(rows, cols, ZR_CKPT_E4M3)
        self.dz = buffer(rows, out_cols, ZR_CKPT_E4M3)
        self.dy = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)
        self.rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        self._packed = self._ran = False

    def pack_weight(self, weight, stream=None) -> None:
        """weight (out_cols x cols, bf16 or fp32) and its transpose, packed."""
        zr_ckpt_pack(weight, self.out_cols, self.cols, self.w, format=self.weight_format, stream=stream)
        zr_ckpt_pack_t(weight, self.out_cols, self.cols, self.w_t, format=self.weight_format, stream=stream)
        self._packed = True

    def forward(self, x, norm_weight, z, residual=None, h=None, bias=None, stream=None) -> None:
        """z (rows x out_cols) of x and the residual, whose sum goes to h."""
        if not self._packed:
            raise ValueError("forward before pack_weight")
        if (bias is not None) != (self.db is not None):
            raise ValueError("the flat gradient has a place for the bias's gradient, and forward has no bias" if bias is None
                             else "forward has a bias, and the layer was made with bias=False")
        zr_rmsnorm_fwd(x, self.rows, self.cols, None, norm_weight, eps=self.eps, residual=residual, h=h,
                       rstd=self.rstd, ckpt_h=self.ckpt_h, ckpt_y=self.ckpt_y, stream=stream)
        zr_ckpt_linear(self.ckpt_y, self.w, self.rows, self.cols, self.out_cols, z, bias=bias,
                       w_format=self.weight_format, workspace=self.scratch, stream=stream)
        self._ran = True

    def backward(self, dz, norm_weight, dx=None, accumulate: bool = False, add_dx: bool = False,
                 stream=None) -> None:
        """The layer's gradients from its output's, dz (rows x out_cols): the
        weights' and the bias's into the flat gradient (added to with accumulate: a
        later micro-step), the input's into dx (added to with add_dx)."""
        if not self._ran:
            raise ValueError("backward before forward")
        rows, cols, out = self.rows, self.cols, self.out_cols
        zr_ckpt_wgrad(dz, self.ckpt_y, rows, out, cols, self.dw, dbias=self.db, accumulate=accumulate,
                      workspace=self.scratch, stream=stream)
        zr_ckpt_pack(dz, rows, out, self.dz, stream=stream)
        zr_ckpt_linear(self.dz, self.w_t, rows, out, cols, self.dy, w_format=self.weight_format,
                       workspace=self.scratch, stream=stream)
        zr_rmsnorm_bwd(self.dy, self.ckpt_h, rows, cols, self.rstd, norm_weight, dx=dx, dweight=self.dw_norm,
                       accumulate=accumulate, add_dx=add_dx, workspace=self.scratch, h_dtype=ZR_CKPT_E4M3,
                       stream=stream)


class ClipAdamW:
    """The optimizer step of K ranks' partitions: their gradients' global norm,
    clipped to max_norm, and AdamW, without a pass for the clipping and without the
    host waiting for the norm.

    grads      : the ranks' fp32 partitions as the reduction leaves them (or any
                 list of gradients, bf16 or fp32)
    params     : fp32 parameters of the same sizes, with exp_avg and exp_avg_sq
    shards     : bf16 copies of the parameters, written with them (or None)
    scale      : the gradients stand for scale * grads (1 / micro-steps, 1 / loss
                 scale)

    step() counts the updates that it enqueues in `steps`. `norm` and `coef` hold the
    last step's; where the gradients are not finite, coef is not, and the step leaves
    the parameters as they are. `left_out`, one int64 on the device, counts those: the
    corrections of the moments go by the updates that were made, steps - left_out. (A
    program that goes on from a checkpoint sets both.) The buffers keep their
    addresses; on another stream than the one that is current when it is made, the
    object has to outlive what step() enqueues.
    """

    def __init__(self, grads: Sequence, params: Sequence, exp_avg: Sequence, exp_avg_sq: Sequence,
                 shards: Optional[Sequence] = None, lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.999,
                 eps: float = 1e-8, weight_decay: float = 0.01, max_norm: float = 1.0, scale: float = 1.0):
        import torch
        self.numels = [g.numel() for g in grads]
        self._tables = [tensor_table(grads, self.numels)] + [tensor_table(xs, self.numels, ZR_FP32)
                                                             for xs in (params, exp_avg, exp_avg_sq)]
        self._shards = None if shards is None else tensor_table(shards, self.numels, ZR_BF16)
        self.lr, self.beta1, self.beta2, self.eps, self.weight_decay = lr, beta1, beta2, eps, weight_decay
        self.max_norm, self.scale = max_norm, scale
        dev = params[0].device
        self.norm, self.coef = torch.zeros(1, device=dev), torch.zeros(1, device=dev)
        self._workspace = torch.empty(zr_grad_norm_workspace_bytes(len(self.numels)), dtype=torch.uint8, device=dev)
        # copied from the host, so that it is there for a first step on any stream
        self.steps, self.left_out = 0, torch.zeros(1, dtype=torch.int64).to(dev)

    def step(self, lr: Optional[float] = None, stream=None) -> None:
        """One update, at rate lr (default: the object's)."""
        g, p, m, v = self._tables
        zr_grad_norm(g, self.numels, self.norm, self.coef, max_norm=self.max_norm, scale=self.scale,
                     workspace=self._workspace, stream=stream)
        zr_adamw(g, self.numels, p, m, v, self.steps + 1, self.lr if lr is None else lr, beta1=self.beta1,
                 beta2=self.beta2, eps=self.eps, weight_decay=self.weight_decay, shards=self._shards,
                 coef=self.coef, left_out=self.left_out, stream=stream)
        self.steps += 1
