"""Batches with shared prefixes, and decoder tokens against encoders: workloads,
runs through the library, references from the oracle."""
import numpy as np
import torch

from _harness import Guarded, GpuRun, assert_attention_close, kvq, oracle_cache, oracle_reference
from int8_kv_cache_reshape_gb300 import workloads as W


def shared_workload(prefix_lens, of, own, new, Hq, Hkv, D, block, dtype, seed, **kw):
    """Request r begins with prefix of[r] (-1: none), then own[r] keys of its
    own, the last new[r] of them queries.  Whole blocks of a prefix are shared,
    the rest of it is written by each request, with the same rows."""
    L = [own[r] + (prefix_lens[p] if p >= 0 else 0) for r, p in enumerate(of)]
    wl = W.custom("shared", list(new), L, Hq, Hkv, D, block, dtype, seed, extra_blocks=2,
                  token_scale_range=(0.2, 5.0) if "per_token" in dtype else None, **kw)
    first = {}
    for r, p in enumerate(of):
        if p < 0:
            continue
        mine = (wl.token_req == r) & (wl.token_pos < prefix_lens[p])
        if p not in first:
            first[p] = (r, wl.key[mine].clone(), wl.value[mine].clone())
            continue
        wl.key[mine], wl.value[mine] = first[p][1], first[p][2]
        whole = prefix_lens[p] // block
        wl.block_table[r, :whole] = wl.block_table[first[p][0], :whole]
        wl.slot_mapping[mine & (wl.token_pos < whole * block)] = -1
    wl.prefix_lens, wl.of = list(prefix_lens), list(of)
    return wl


class SharedRun(GpuRun):
    """A workload through a schedule with shared prefixes."""

    def schedule(self):
        wl = self.wl
        return kvq().get_shared_prefix_metadata(
            wl.num_req, wl.heads_q, wl.heads_kv, wl.head_dim, wl.seq_lens_t, wl.query_start_loc, wl.prefix_lens,
            wl.of, wl.window, wl.kv_cache_dtype)

    def attention(self, sched=None, workspace=None):
        wl, k = self.wl, kvq()
        own = sched is None
        sched = sched or self.schedule()
        # (NaN: a partial row that is read without having been written shows)
        ws = workspace or Guarded((max(sched.workspace_bytes, 1),), torch.uint8, 0xFF, self.q.device)
        k.attention_with_kv_cache(sched, self.q, self.kc, self.vc, self.qsl, self.sl, self.bt, wl.sm_scale, wl.causal,
                                  wl.window, wl.soft_cap, wl.k_scale, wl.v_scale, self.out, ws.t, wl.kv_cache_dtype,
                                  wl.heads_kv, alibi_slopes=self.alibi, sinks=self.sinks)
        torch.cuda.synchronize()
        sched.check_device()
        ws.check("workspace")
        self._out.check("output")
        self._kc.check("key cache (read only)")
        self._vc.check("value cache (read only)")
        self.rect, self.sched_info = sched.rect_info(), sched.info()
        if own:
            sched.close()
        return self


class CrossRun(SharedRun):
    def schedule(self):
        wl = self.wl
        return kvq().get_cross_attention_metadata(wl.num_req, wl.heads_q, wl.heads_kv, wl.head_dim, wl.seq_lens_t,
                                                  wl.query_start_loc, wl.kv_cache_dtype)


def compare(g, what, tokens=None, cache=None):
    """The output against the oracle, at the bound of a binary32 evaluation
    (_harness); rows of requests without keys are zero."""
    wl = g.wl
    kc, vc = cache or oracle_cache(wl)
    req = np.repeat(np.arange(wl.num_req), wl.query_lens)
    live = np.asarray(wl.seq_lens)[req] > 0
    tokens = np.flatnonzero(live) if tokens is None else np.asarray(tokens)
    got = g.out_f32()
    assert not got[~live].any(), f"{what}: rows without keys"
    ref, bound = oracle_reference(wl, kc, vc, tokens=tokens, alibi_slopes=g.alibi_np, sinks=g.sinks_np)
    return assert_attention_close(got[tokens], ref, what, bound)
