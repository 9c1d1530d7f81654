"""Decode-step runtime over a stack of attention layers.

Holds, per layer, the device state of the rotated int4 path (page pool, block table,
M_q/M_k) or of the FP8 sliding-window path (ring), plus one shared workspace and error
word; `decode_step` runs every layer of one decode step through the C ABI, in model
order (Kolibri-1: 50 layers, every fifth one full attention; "Serving Kolibri-1 with a
4-bit KV cache", section "What we do"). Torch is used for device memory only.
"""

from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

from . import (HEAD_DIM, MAX_CACHES, PAGE_SIZE, alloc_fp8_ring, alloc_int4_cache, alloc_mass_workspace, alloc_prompt_mass_workspace,
               alloc_prompt_workspace, alloc_token_mass, alloc_tree_workspace, alloc_workspace, kvq_build_rotation,
               kvq_decode_attn_fp8_swa, kvq_decode_attn_int4, kvq_evict_int4, kvq_fold_qk, kvq_fold_qk_fwht, kvq_fp8_append,
               kvq_mass_attn_int4, kvq_mass_start, kvq_prompt_attn, kvq_prompt_mass, kvq_rotate_quant_append,
               kvq_tree_attn_fp8_swa, kvq_tree_attn_int4, kvq_tree_commit_fp8, kvq_tree_commit_int4, kvq_window_attn_int4)


@dataclass
class Int4Layer:
    tensors: dict
    cache: object
    Mq: torch.Tensor  # folded query matrix, or the FWHT multipliers w_q
    Mk: torch.Tensor  # R, or the FWHT multipliers w_k = s
    R: np.ndarray
    fwht: bool = False
    window: int = 0       # > 0: rows see the last `window` tokens and the first `sinks` (set_int4_window)
    sinks: int = 0
    held: dict = None     # keep_mass: what the cache's slots have gathered, and its descriptor
    mass: object = None
    observed: bool = False  # observe_prompt sets masses of this layer


@dataclass
class SwaLayer:
    tensors: dict
    ring: object
    k_scale: float
    v_scale: float
    window: int


class DecodeStack:
    """Layers l = 0..n_layers-1; layer l is full attention (int4) when l % full_every == full_every-1."""

    def __init__(self, B, Hq, Hkv, S, max_pages, n_layers=1, full_every=1, ring_capacity=576, window=513,
                 swa_k_scale=1.0, swa_v_scale=1.0, page_perm=None, device="cuda"):
        self.B, self.Hq, self.Hkv, self.S = B, Hq, Hkv, S
        self.max_pages = max_pages
        self.device = device
        self.layers = []
        for l in range(n_layers):
            if l % full_every == full_every - 1:
                npages = B * max_pages
                perm = page_perm(l, npages) if page_perm is not None else np.arange(npages, dtype=np.int32)
                bt = torch.from_numpy(np.ascontiguousarray(perm.reshape(B, max_pages), dtype=np.int32))
                tensors, cache = alloc_int4_cache(npages, Hkv, bt, device)
                self.layers.append(Int4Layer(tensors, cache, None, None, None))
            else:
                tensors, ring = alloc_fp8_ring(B, Hkv, ring_capacity, device)
                self.layers.append(SwaLayer(tensors, ring, swa_k_scale, swa_v_scale, window))
        self.workspace = alloc_workspace(B, S, Hq, Hkv, device)
        self.mass_workspace = None  # keep_mass
        self.dev_err = torch.zeros(1, dtype=torch.int32, device=device)

    def int4_layers(self):
        return [i for i, L in enumerate(self.layers) if isinstance(L, Int4Layer)]

    def swa_layers(self):
        return [i for i, L in enumerate(self.layers) if isinstance(L, SwaLayer)]

    def set_int4_params(self, l, rot_seed, g_q, g_k, rotate=True, prologue="matrix"):
        """Build R from the seed and fold the gains (host), upload M_q and M_k. rotate=False folds
        R = I instead: the unrotated int4 baseline (M_q = diag(g_q g_k), M_k = I).
        prologue="fwht": the same rotation through the fast Walsh-Hadamard prologue (uploads the
        multipliers w_q = s g_q g_k and w_k = s); set it before filling the layer's cache."""
        L = self.layers[l]
        if prologue == "fwht":
            R, s = kvq_build_rotation(rot_seed)
            wq, wk = kvq_fold_qk_fwht(s, g_q, g_k)
            L.R, L.fwht = R, True
            L.Mq = torch.from_numpy(wq).to(self.device)
            L.Mk = torch.from_numpy(wk).to(self.device)
            return
        assert prologue == "matrix", prologue
        R = kvq_build_rotation(rot_seed)[0] if rotate else np.eye(HEAD_DIM, dtype=np.float32)
        Mq, Mk = kvq_fold_qk(R, g_q, g_k)
        L.R, L.fwht = R, False
        L.Mq = torch.from_numpy(Mq).to(self.device)
        L.Mk = torch.from_numpy(Mk).to(self.device)

    def append_int4(self, l, k, v, seq_ids, positions, stream=None, slots=None, fresh=None):
        """Tokens into the cache of int4 layer l, each at its position; in a layer that keeps mass at slots (None: the
        positions), where evictions have made the two differ. There the slots' masses start with the tokens: a slot that holds
        another number than the token's gets that number, and no mass. fresh: so does every slot, whatever its number (a new
        session in a row that another has used); None: unless prompts of this layer are observed, where the call that
        observes them sets the masses, before this one or after it."""
        L = self.layers[l]
        if L.mass is None or slots is None:
            slots = positions
        kvq_rotate_quant_append(L.cache, L.Mk, k, v, seq_ids, slots, self.dev_err, stream=stream, fwht=L.fwht)
        if L.mass is not None:
            lists = (x if x.shape[0] == k.shape[0] else x[:k.shape[0]] for x in (seq_ids, slots, positions))
            kvq_mass_start(L.mass, *lists, self.dev_err, fresh=not L.observed if fresh is None else fresh, stream=stream)

    def prefill_int4(self, l, ctx, fill, chunk_tokens=16384, bf16=True):
        """Append positions 0..ctx[b]-1 of every sequence; fill(b, pos0, T, k_out, v_out) writes the
        pre-norm keys and values of those positions into device buffers [T, Hkv, 128]."""
        dt = torch.bfloat16 if bf16 else torch.float32
        kbuf = torch.empty((chunk_tokens, self.Hkv, HEAD_DIM), dtype=dt, device=self.device)
        vbuf = torch.empty_like(kbuf)
        for b in range(self.B):
            for p0 in range(0, int(ctx[b]), chunk_tokens):
                T = min(chunk_tokens, int(ctx[b]) - p0)
                fill(b, p0, T, kbuf, vbuf)
                seq = torch.full((T,), b, dtype=torch.int32, device=self.device)
                pos = torch.arange(p0, p0 + T, dtype=torch.int32, device=self.device)
                self.append_int4(l, kbuf[:T], vbuf[:T], seq, pos)

    def decode_layer(self, l, q, ctx, out, k_new=None, v_new=None, q_rot_out=None, stream=None, positions=None):
        """ctx: the cached tokens; positions: the tokens that the sequences have had, where some layers have evicted any
        (those that keep mass hold ctx tokens, all others every one)."""
        L = self.layers[l]
        if isinstance(L, Int4Layer) and (L.mass is not None or L.window) and q_rot_out is not None:
            raise ValueError("q_rot_out: of layers that see their whole cache only")
        if isinstance(L, Int4Layer) and L.mass is not None:
            kvq_mass_attn_int4(L.cache, L.mass, L.Mq, L.Mk, q, ctx, ctx if positions is None else positions, out,
                               self.mass_workspace, self.dev_err, k_new=k_new, v_new=v_new, stream=stream, fwht=L.fwht)
            return
        ctx = ctx if positions is None else positions
        if isinstance(L, Int4Layer) and L.window:
            kvq_window_attn_int4(L.cache, L.Mq, L.Mk, q, ctx, L.window, L.sinks, out, self.workspace, self.dev_err,
                                 k_new=k_new, v_new=v_new, stream=stream, fwht=L.fwht)
        elif isinstance(L, Int4Layer):
            kvq_decode_attn_int4(L.cache, L.Mq, L.Mk, q, ctx, out, self.workspace, self.dev_err, k_new=k_new,
                                 v_new=v_new, q_rot_out=q_rot_out, stream=stream, fwht=L.fwht)
        else:
            kvq_decode_attn_fp8_swa(L.ring, q, ctx, L.window, L.k_scale, L.v_scale, out, self.workspace,
                                    self.dev_err, k_new=k_new, v_new=v_new, stream=stream)

    def decode_step(self, qs, ctx, outs, k_news=None, v_news=None, stream=None, positions=None):
        """One decode step over all layers: qs[l], outs[l], k_news[l], v_news[l] per layer; positions as decode_layer."""
        for l in range(len(self.layers)):
            self.decode_layer(l, qs[l], ctx, outs[l], None if k_news is None else k_news[l],
                              None if v_news is None else v_news[l], stream=stream, positions=positions)

    # ---- around decoding

    def _alloc_for(self, stream, alloc, *sizes):
        """A workspace (or what layers keep) allocated in the order of the stream that will use it (None: the current one; else a
        stream or its raw handle), so that the allocator hands its memory to nothing else before that stream is done with it."""
        if stream is None:
            return alloc(*sizes, self.device)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream)
        with torch.cuda.stream(stream):
            return alloc(*sizes, self.device)

    def prompt_layer(self, l, q, k, v, cu_seqlens, out, workspace=None, stream=None):
        """Attention of whole prompts, packed end to end, in layer l (windowed in a sliding-window layer);
        q, k and v as kvq_prompt_attn takes them. The keys and values go into the cache by
        append_prompt."""
        L = self.layers[l]
        if workspace is None:  # (of 256 bytes, see kvq.h)
            workspace = self._alloc_for(stream, alloc_prompt_workspace, q.shape[0], cu_seqlens.shape[0] - 1, self.Hq, self.Hkv)
        kvq_prompt_attn(q, k, v, cu_seqlens, out, workspace, self.dev_err, window=L.window,
                        sinks=L.sinks if isinstance(L, Int4Layer) else 0, stream=stream)

    def append_prompt(self, l, k, v, seq_ids, positions, stream=None, slots=None, fresh=None):
        """Keys (pre-norm in a full-attention layer) and values of prompt tokens into layer l's cache. A ring keeps
        the last `capacity` positions of a sequence: pass no more of them in one call. slots, fresh: of layers that keep
        mass, as append_int4 takes them."""
        L = self.layers[l]
        if isinstance(L, Int4Layer):
            self.append_int4(l, k, v, seq_ids, positions, stream=stream, slots=slots, fresh=fresh)
        else:
            kvq_fp8_append(L.ring, k, v, seq_ids, positions, L.k_scale, L.v_scale, self.dev_err, stream=stream)

    def tree_layer(self, l, q, ctx, tree_mask, out, workspace, k_new=None, v_new=None, stream=None):
        """Attention of every sequence's tree of drafted tokens in layer l (workspace: alloc_tree_workspace)."""
        L = self.layers[l]
        if isinstance(L, Int4Layer) and (L.window or L.mass is not None):
            raise ValueError("a tree sees its layer's whole cache and keeps no mass")
        if isinstance(L, Int4Layer):
            kvq_tree_attn_int4(L.cache, L.Mq, L.Mk, q, ctx, tree_mask, out, workspace, self.dev_err, k_new=k_new,
                               v_new=v_new, stream=stream, fwht=L.fwht)
        else:
            kvq_tree_attn_fp8_swa(L.ring, q, ctx, tree_mask, L.window, L.k_scale, L.v_scale, out, workspace,
                                  self.dev_err, k_new=k_new, v_new=v_new, stream=stream)

    def tree_step(self, qs, ctx, tree_mask, outs, k_news=None, v_news=None, workspace=None, stream=None):
        """One verify step over all layers: qs[l], outs[l], k_news[l], v_news[l] per layer."""
        if workspace is None:
            workspace = self._alloc_for(stream, alloc_tree_workspace, qs[0].shape[0], qs[0].shape[1], self.Hq, self.Hkv)
        for l in range(len(self.layers)):
            self.tree_layer(l, qs[l], ctx, tree_mask, outs[l], workspace, None if k_news is None else k_news[l],
                            None if v_news is None else v_news[l], stream=stream)

    def commit_tree(self, ctx, path, n_accept, ctx_out, stream=None):
        """The accepted branch of every tree becomes context in all layers; ctx_out: the new lengths. (Layers that keep mass
        take no trees: records would move without their masses, and by lengths that are not theirs after an eviction.)"""
        if self.mass_layers():
            raise ValueError("a layer that keeps mass takes no trees, and commits none")
        for commit, layers in ((kvq_tree_commit_int4, [self.layers[l].cache for l in self.int4_layers()]),
                               (kvq_tree_commit_fp8, [self.layers[l].ring for l in self.swa_layers()])):
            for i in range(0, len(layers), MAX_CACHES):  # as many layers as a call takes
                commit(layers[i:i + MAX_CACHES], ctx, path, n_accept, self.dev_err, ctx_out=ctx_out, stream=stream)
                ctx_out = None  # written once

    # ---- caches held to a size

    def set_int4_window(self, l, window, sinks=0):
        """Rows of full-attention layer l see the last `window` tokens and the first `sinks`, in prompts and decode steps
        (window 0: all again)."""
        L = self.layers[l]
        if not isinstance(L, Int4Layer) or L.mass is not None or window < 0 or sinks < 0:
            raise ValueError("a window is of an int4 layer that keeps no mass, its sizes not negative")
        L.window, L.sinks = window, sinks

    def keep_mass(self, layers=None, stream=None):
        """From here on the int4 layers `layers` (None: all without a window) keep what their slots gather, and can evict. Layers
        that do already go on, and the workspace of the steps stays where it is, so that steps in flight and captured ones may.
        stream: the one that prompts and steps will run on (None: the current one); what they need is laid out in its order."""
        layers = [l for l in self.int4_layers() if not self.layers[l].window] if layers is None else layers
        if any(not isinstance(self.layers[l], Int4Layer) or self.layers[l].window for l in layers):
            raise ValueError("mass is kept by int4 layers without a window")
        if self.mass_workspace is None:
            self.mass_workspace = self._alloc_for(stream, alloc_mass_workspace, self.B, self.Hq, self.Hkv, self.max_pages * PAGE_SIZE)
        for l in set(layers) - set(self.mass_layers()):
            self.layers[l].held, self.layers[l].mass = self._alloc_for(stream, alloc_token_mass, self.B, self.Hkv, self.max_pages)

    def mass_layers(self):
        return [l for l in self.int4_layers() if self.layers[l].mass is not None]

    def observe_prompt(self, l, q, k, cu_seqlens, rows, seq_ids=None, workspace=None, stream=None):
        """Layer l's mass starts from the weights of each prompt's last `rows` rows; q and k as prompt_layer takes them."""
        if l not in self.mass_layers():
            raise ValueError("a layer that keeps no mass")
        self.layers[l].observed = True
        if workspace is None:
            workspace = self._alloc_for(stream, alloc_prompt_mass_workspace, q.shape[0], cu_seqlens.shape[0] - 1, self.Hq, self.Hkv, rows)
        kvq_prompt_mass(q, k, cu_seqlens, rows, self.layers[l].mass, workspace, self.dev_err, seq_ids=seq_ids, stream=stream)

    def evict(self, ctx, seen, budget, sinks, recent, ctx_out, stream=None):
        """Every layer that keeps mass evicts down to `budget` tokens a sequence and KV head (kvq_evict_int4); ctx_out: the
        new lengths."""
        layers = [self.layers[l] for l in self.mass_layers()]
        if not layers:
            raise ValueError("no layer keeps mass")
        for i in range(0, len(layers), MAX_CACHES):  # as many layers as a call takes
            some = layers[i:i + MAX_CACHES]
            kvq_evict_int4([L.cache for L in some], [L.mass for L in some], ctx, seen, budget, sinks, recent, self.dev_err,
                           ctx_out=None if i else ctx_out, stream=stream)

    def read_error(self) -> int:
        return int(self.dev_err.item())


def pages_needed(ctx_max: int, extra_positions: int) -> int:
    return (ctx_max + extra_positions + PAGE_SIZE - 1) // PAGE_SIZE
