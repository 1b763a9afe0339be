"""A stack of GCN / GraphSAGE-mean layers over one prepared graph.

Owns the per-layer device buffers (saved activations, gradients, one
shared workspace) and runs forward / backward through the C ABI layer
calls; no arithmetic happens here.  Layer l uses ReLU except the last
(AdaQP Sec. 2.1 layer form with sigma = ReLU on hidden layers).

Between the hidden layers a stack may normalize and drop features, and it
may end in a class head (gq_train.h; the pages describe neither):

    hidden layer l:  H = A W;  input of layer l + 1 = drop(relu(norm(H))), norm
                     over a node's row (layer) or over each graph of a batch and
                     groups of channels (group)
                     (without norm: drop(relu(H)))
    class head:      loss = mean cross entropy of softmax(H_last Wc^T) over
                     the labelled nodes; scores = H_last Wc^T of 8-bit integers
    optimizer:       AdamW on the stack's gradient buffers
"""
from __future__ import annotations

import torch

from . import (ACT_NONE, ACT_RELU, COEF_GCN, DROPOUT_SEED_TAG, F32, AdamW, GQError, Graph, Workspace, dropout,
               gcn_layer_bwd, gcn_layer_fwd, group_norm_bwd, group_norm_fwd, layer_norm_bwd, layer_norm_fwd, lib,
               linear_i8, linear_xent, to_bf16)

# stages traced per call (see gq_gcn_layer_fwd / gq_gcn_layer_bwd)
FWD_STAGES = ("quantize", "aggregate", "update_gemm")
BWD_STAGES = ("dz", "dw_gemm", "da_gemm", "quantize_bwd", "aggregate_t")


def launches_fwd(bits: int) -> int:
    """Kernels one gq_gcn_layer_fwd call launches: [quantize] + aggregate
    + W transpose + GEMM."""
    return (1 if bits < 32 else 0) + 3


def launches_bwd(bits: int, need_dinput: bool, dz_given: bool = False) -> int:
    """[dZ] + weight GEMM + split reduction [+ W convert + dA GEMM +
    [quantize] + transposed aggregate]."""
    n = 2 if dz_given else 3
    if need_dinput:
        n += 3 + (1 if bits < 32 else 0)
    return n


class GCNStack:
    """norm: True or "layer" for layer normalization, "group" for group
    normalization behind every hidden layer (its weights are the `norms` of
    forward and backward, a (gamma, beta) pair per hidden layer; gradients in
    dgamma, dbeta).  "group" takes groups, and, where the graph is a batch of
    graphs, ptr, the int64 offsets of their nodes (on the stack's device, rising from 0 to
    the number of nodes: a node outside every graph would have no features; read
    once, here), and max_rows, the largest one's number of nodes.  p: dropout rate of the hidden
    layers' outputs (training passes only).  classes: width of the class
    head behind the last layer (loss_and_grad, loss; gradient in dWc).  With
    norm or p the hand-off of dZ between layers is theirs, and fuse_dz does
    not apply."""

    def __init__(self, g: Graph, widths, mask: torch.Tensor | None, coef: int = COEF_GCN,
                 device="cuda", keep_dA: bool = False, fuse_dz: bool = True, norm: bool | str = False, p: float = 0.0,
                 classes: int = 0, groups: int = 1, ptr: torch.Tensor | None = None, max_rows: int = 0):
        if not 0.0 <= p <= 1.0 or classes < 0:
            raise GQError("p must lie in [0, 1] and classes must not be negative")
        if norm not in (True, False, None, "layer", "group"):
            raise GQError(f'norm must be "layer", "group", True (layer) or False, got {norm!r}')
        self.grouped = grouped = norm == "group"
        if not grouped and (groups != 1 or ptr is not None or max_rows):
            raise GQError('groups, ptr and max_rows go with norm="group"')
        if grouped and (groups < 1 or max_rows < 0 or any(w % groups for w in widths[1:-1])):
            raise GQError(f"every hidden width must be a multiple of the {groups} groups, max_rows not negative")
        if grouped and ptr is not None:
            if ptr.dtype != torch.int64 or ptr.dim() != 1 or ptr.numel() < 1 or ptr.device.type != torch.device(device).type:
                raise GQError("ptr must be an int64 vector of node offsets on the stack's device")
            offsets = ptr.cpu()
            if offsets[0] != 0 or offsets[-1] != g.n or (offsets[1:] < offsets[:-1]).any():
                raise GQError(f"ptr must rise from 0 to the graph's {g.n} nodes")
        norm = bool(norm)
        self.groups, self.ptr, self.max_rows = groups, ptr, max_rows
        self.norm, self.p, self.classes = norm, float(p), classes
        self.g = g
        self.widths = tuple(widths)
        self.L = len(widths) - 1
        self.mask = mask
        self.coef = coef
        n = g.n
        self.ws = Workspace(device)
        r8 = lambda x: (x + 7) // 8 * 8
        self.A = [torch.empty(n, r8(widths[l]), dtype=torch.bfloat16, device=device) for l in range(self.L)]
        self.H = [torch.empty(n, widths[l + 1], dtype=torch.float32, device=device) for l in range(self.L)]
        self.dH = [torch.empty(n, widths[l], dtype=torch.float32, device=device) for l in range(self.L)]
        self.dW = [torch.empty(widths[l], widths[l + 1], dtype=torch.float32, device=device) for l in range(self.L)]
        # the backward's dA = dZ W^T of each layer (the messages it quantizes), kept on request
        self.dA = [torch.empty(n, widths[l], dtype=torch.float32, device=device) if keep_dA else None
                   for l in range(self.L)]
        # fuse_dz: the transposed aggregation of layer l writes layer l-1's dZ
        # (bf16, ReLU gate applied) instead of an fp32 gradient, which layer
        # l-1 then takes as its dZ
        fuse_dz = fuse_dz and not norm and p == 0.0
        self.fuse_dz = fuse_dz
        self.dZ = [torch.empty(n, r8(widths[l + 1]), dtype=torch.bfloat16, device=device)
                   if fuse_dz and l < self.L - 1 else None for l in range(self.L)]
        # with fuse_dz: [H[l] > 0] as bits (written by layer l's forward GEMM),
        # the gate layer l+1's transposed aggregation applies to dZ[l]
        self.Rb = [torch.empty(n, (widths[l + 1] + 31) // 32, dtype=torch.int32, device=device)
                   if fuse_dz and l < self.L - 1 else None for l in range(self.L)]
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        # what stands between the hidden layers: the next layer's input, the
        # row statistics, the ReLU bits, the bf16 dZ that normalization's
        # backward pass hands the layer, and the dropout seeds of the last
        # forward pass
        hidden = range(self.L - 1)
        e32 = lambda *shape: torch.empty(*shape, dtype=torch.float32, device=device)
        self.N = [e32(n, widths[l + 1]) if norm or p > 0.0 else None for l in hidden]
        stats = (n,) if not grouped else (1 if ptr is None else ptr.numel() - 1, groups)
        self.mean = [e32(*stats) if norm else None for l in hidden]
        self.rstd = [e32(*stats) if norm else None for l in hidden]
        self.dgamma = [e32(widths[l + 1]) if norm else None for l in hidden]
        self.dbeta = [e32(widths[l + 1]) if norm else None for l in hidden]
        if norm and not grouped:  # group normalization makes its ReLU's derivative again, and its gradient in place
            for l in hidden:
                self.Rb[l] = torch.empty(n, (widths[l + 1] + 31) // 32, dtype=torch.int32, device=device)
                self.dZ[l] = torch.empty(n, r8(widths[l + 1]), dtype=torch.bfloat16, device=device)
        self._drop = [None] * (self.L - 1)
        # of the latest forward pass: it dropped, it had normalization weights,
        # the last layer's dZ is the head's gradient on it
        self._training = self._weighted = self._graded = False
        if classes:
            d = widths[self.L]
            self.Hb = torch.empty(n, r8(d), dtype=torch.bfloat16, device=device)
            self.node_loss = e32(n)
            self.dWc = torch.empty_strided((classes, d), (r8(d), 1), dtype=torch.bfloat16, device=device)
            self.dZ[self.L - 1] = torch.empty(n, r8(d), dtype=torch.bfloat16, device=device)
            self.ws_head = Workspace(device)
        L = lib()
        self.ws.get(max([int(L.gq_gcn_layer_workspace_bytes(g.ref, widths[l], widths[l + 1], 2))
                         for l in range(self.L)] +
                        [int(L.gq_layer_norm_bwd_workspace_bytes(n, widths[l + 1])) for l in hidden
                         if norm and not grouped] +
                        [self._group_ws(l, b) for l in hidden for b in (0, 1) if grouped]))
        if classes:
            self.ws_head.get(int(L.gq_linear_xent_workspace_bytes(n, widths[self.L], classes, 1)))

    def _group_ws(self, l, backward):
        """Workspace of hidden layer l's group normalization."""
        return int(lib().gq_group_norm_workspace_bytes(self.g.n, self.widths[l + 1], self.groups, F32,
                                                       self.mean[l].shape[0], self.max_rows, backward))

    def act(self, l: int) -> int:
        return ACT_RELU if l < self.L - 1 and not self.norm else ACT_NONE

    def _norm_of(self, norms, l):
        if norms is None:
            return None, None
        if len(norms) != self.L - 1:
            raise GQError(f"norms: one (gamma, beta) pair for each of the {self.L - 1} hidden layers")
        return norms[l]

    def forward(self, X: torch.Tensor, Ws, bits: int, seeds, events=None, norms=None, training: bool = True):
        """The last layer's output.  training = False leaves dropout out; it
        overwrites what a backward pass needs, so that with p > 0 one follows
        a training pass only."""
        self._training = training
        self._graded = False
        self._weighted = norms is not None
        h = X
        for l in range(self.L):
            ev = None if events is None else events[l]
            hidden = l < self.L - 1
            gcn_layer_fwd(self.g, h, Ws[l], self.mask, bits, seeds[l], self.act(l), coef=self.coef, ws=self.ws,
                          A_save=self.A[l], H_out=self.H[l], dev_err=self.err, events=ev,
                          relu_bits=self.Rb[l] if self.fuse_dz else None)
            h = self.H[l]
            if not hidden:
                continue
            p = self.p if training else 0.0
            # the layer's quantizer draws its noise from the same seed
            seed = self._drop[l] = seeds[l] ^ DROPOUT_SEED_TAG
            if self.grouped:
                gamma, beta = self._norm_of(norms, l)
                h, _, _ = group_norm_fwd(h, self.groups, self.ptr, gamma, beta, act=ACT_RELU, max_rows=self.max_rows,
                                         out=self.N[l], mean=self.mean[l], rstd=self.rstd[l], ws=self.ws)
                if p > 0.0:
                    dropout(h, p, seed, out=h)
            elif self.norm:
                gamma, beta = self._norm_of(norms, l)
                layer_norm_fwd(h, gamma, beta, act=ACT_RELU, p=p, seed=seed, out=self.N[l], mean=self.mean[l],
                               rstd=self.rstd[l], relu_bits=self.Rb[l])
                h = self.N[l]
            elif p > 0.0:
                h = dropout(h, p, seed, out=self.N[l])
        return h

    def backward(self, dY: torch.Tensor | None, Ws, bits: int, seeds, need_input_grad: bool = False, events=None,
                 norms=None):
        """Weight gradients from dY, or, with dY None, from the dZ that
        loss_and_grad left for the last layer (refused where it has not run
        since the latest forward pass)."""
        if dY is None and not self.classes:
            raise GQError("backward needs dY: the stack has no class head")
        if dY is None and not self._graded:
            raise GQError("backward without dY follows loss_and_grad on the latest forward pass")
        if self.p > 0.0 and not self._training:
            raise GQError("backward follows a training forward pass")
        if self.norm and self._weighted != (norms is not None):
            raise GQError("norms: backward takes the normalization weights of the forward pass, if it had any")
        g = dY
        for l in reversed(range(self.L)):
            need = need_input_grad or l > 0
            ev = None if events is None else events[l]
            top = l == self.L - 1
            dz_in = self.dZ[l] if not top or dY is None else None  # made above this layer, else None
            fuse = self.fuse_dz and l > 0                    # layer l makes layer l-1's dZ
            gcn_layer_bwd(self.g, None if dz_in is not None else g, self.A[l],
                          None if dz_in is not None else self.H[l], Ws[l], self.mask, bits, seeds[l],
                          self.act(l), need, coef=self.coef, ws=self.ws, dW=self.dW[l],
                          dH_in=self.dH[l] if need and not fuse else None,
                          dA_save=self.dA[l] if need else None, dev_err=self.err, events=ev, dZ_in=dz_in,
                          gate_in=self.Rb[l - 1] if fuse else None, dZ_prev=self.dZ[l - 1] if fuse else None)
            g = self.dH[l]
            if l == 0:
                continue
            if self.grouped:
                gamma, beta = self._norm_of(norms, l - 1)
                if self.p > 0.0:
                    dropout(g, self.p, self._drop[l - 1], out=g)
                group_norm_bwd(g, self.H[l - 1], self.groups, self.mean[l - 1], self.rstd[l - 1], self.ptr, gamma, beta,
                               act=ACT_RELU, max_rows=self.max_rows, dX=g, dgamma=self.dgamma[l - 1],
                               dbeta=self.dbeta[l - 1], ws=self.ws)
            elif self.norm:
                gamma, _ = self._norm_of(norms, l - 1)
                layer_norm_bwd(g, self.H[l - 1], self.mean[l - 1], self.rstd[l - 1], gamma, act=ACT_RELU, p=self.p,
                               seed=self._drop[l - 1], relu_bits=self.Rb[l - 1],
                               dX=self.dZ[l - 1][:, :self.widths[l]], dgamma=self.dgamma[l - 1],
                               dbeta=self.dbeta[l - 1], ws=self.ws)
            elif self.p > 0.0:
                dropout(g, self.p, self._drop[l - 1], out=g)
        return self.dW

    def _head(self, Wc, labels, scale, weight, grad):
        if not self.classes or Wc.shape != (self.classes, self.widths[self.L]):
            raise GQError(f"the stack's class head is {self.classes} x {self.widths[self.L]}")
        d = self.widths[self.L]
        to_bf16(self.H[self.L - 1], out=self.Hb)
        return linear_xent(self.Hb[:, :d], Wc, labels, weight, scale, grad=grad, loss=self.node_loss,
                           dX=self.dZ[self.L - 1][:, :d] if grad else None, dW=self.dWc if grad else None,
                           ws=self.ws_head, dev_err=self.err)[0]

    def loss(self, Wc: torch.Tensor, labels: torch.Tensor) -> torch.Tensor:
        """Per-node cross entropy of the head on the latest forward pass's
        output (0 for nodes without a label): the stack's own buffer, which
        the next call of loss or loss_and_grad overwrites."""
        return self._head(Wc, labels, 1.0, None, False)

    def loss_and_grad(self, Wc: torch.Tensor, labels: torch.Tensor, scale: float,
                      weight: torch.Tensor | None = None) -> torch.Tensor:
        """Per-node cross entropy; leaves the gradients of scale *
        sum(weight * loss) in dWc and, for backward(None, ...), in the last
        layer's dZ.  scale: 1 / (number of labelled nodes) for their mean.
        Returns the buffer that loss returns."""
        loss = self._head(Wc, labels, scale, weight, True)
        self._graded = True
        return loss

    def scores(self, Wc: torch.Tensor, scale: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
        """Scores of every node over classes on the latest forward pass's
        output: H_last Wc^T with both quantized to 8 bits, Wc and scale as
        quantize_i8 left them (any number of classes; no head is needed)."""
        if getattr(self, "ws_scores", None) is None:
            self.ws_scores = Workspace(self.H[0].device)
        return linear_i8(self.H[self.L - 1], Wc, scale, out=out, ws=self.ws_scores, dev_err=self.err)

    def optimizer(self, Ws, norms=None, Wc: torch.Tensor | None = None, **kw) -> AdamW:
        """An AdamW over the weights, the normalization weights (where forward
        is given them) and the class head's, whose gradients are the buffers that
        backward and loss_and_grad write: after them, step() updates all in place.
        kw: AdamW's arguments (lr, betas, eps, weight_decay, state_bits, ...)."""
        params, grads = list(Ws), list(self.dW)
        if len(params) != self.L:
            raise GQError(f"Ws: one weight matrix for each of the {self.L} layers")
        if norms is not None:
            if not self.norm or len(norms) != self.L - 1:
                raise GQError(f"norms: one (gamma, beta) pair for each of the {self.L - 1} hidden layers of a stack with norm")
            for l, pair in enumerate(norms):
                params += pair
                grads += [self.dgamma[l], self.dbeta[l]]
        if Wc is not None:
            if not self.classes or Wc.shape != self.dWc.shape:
                raise GQError("Wc: the weights of the stack's class head")
            params.append(Wc)
            grads.append(self.dWc)
        return AdamW(params, grads=grads, **kw)

    def launches(self, bits: int, need_input_grad: bool = False) -> int:
        """Kernels of one forward and backward pass (from the class head's
        gradient where there is a head), the head's own not counted."""
        n = sum(launches_fwd(bits) + launches_bwd(bits, need_input_grad or l > 0, self.dZ[l] is not None)
                for l in range(self.L))
        if self.grouped:  # one pass each way, or three, and the column sums; dropout one each
            return n + sum((3 if self._group_ws(l, 0) else 1) + (4 if self._group_ws(l, 0) else 2) +
                           (2 if self.p > 0.0 else 0) for l in range(self.L - 1))
        # normalization: one forward, the pass and its column sums backward; dropout alone: one each
        return n + (self.L - 1) * (3 if self.norm else 2 if self.p > 0.0 else 0)
