// Sequences, masks and cache addressing shared by the paged-attention kernels.
#pragma once

#include "kda_internal.cuh"

namespace kda {

struct Seq {
  int bos;   // first token of the sequence in the packed token axis
  int len;   // new tokens
  int kv;    // keys of the sequence, the new tokens' included
  int pos0;  // position of its first new token (negative: more new tokens than keys)
  int list, pre;  // the prefix that its items take along with its own keys, and its keys (list < 0:
                  // none; kda_paged_plan.cuh)
};

// Lists of keys: those of the shared prefixes, which all tokens of a group of sequences see, and
// behind them the sequences' own.  List i < groups is a prefix, list groups + n is sequence n's.
__device__ __forceinline__ int lists(const PagedArgs& a) { return a.groups + a.N; }
// Block table row of a list.
__device__ __forceinline__ const int32_t* table_of(const PagedArgs& a, int i) {
  return i < a.groups ? a.prefix_table + (long long)i * a.max_prefix_pages
                      : a.block_table + (long long)(i - a.groups) * a.max_pages;
}
// Raw offsets and key count of a list.
__device__ __forceinline__ void raw_seq(const PagedArgs& a, int i, int& lo, int& hi, int& kv) {
  if (i < a.groups) {
    lo = a.cu_seqlens[min(max(a.cu_groups[i], 0), a.N)];
    hi = a.cu_seqlens[min(max(a.cu_groups[i + 1], 0), a.N)];
    kv = a.prefix_lens[i];
  } else {
    lo = a.cu_seqlens[i - a.groups];
    hi = a.cu_seqlens[i - a.groups + 1];
    kv = a.kv_lens[i - a.groups];
  }
}

// From a list's raw offsets and key count.  All of a prefix is in its tokens' past: they are given
// the position of its last key (positions behind it are clamped to it where they count).
__device__ __forceinline__ Seq make_seq(const PagedArgs& a, int lo, int hi, int kv, bool prefix) {
  Seq s;
  lo = min(max(lo, 0), a.total_T);
  hi = min(max(hi, lo), a.total_T);
  s.bos = lo;
  s.len = hi - lo;
  const long long cap = (long long)(prefix ? a.max_prefix_pages : a.max_pages) * a.page_size;
  s.kv = (int)min((long long)max(kv, 0), a.num_pages > 0 ? cap : 0ll);
  s.pos0 = s.kv - (prefix ? 1 : s.len);
  s.list = -1;
  s.pre = 0;
  return s;
}
__device__ __forceinline__ Seq load_seq(const PagedArgs& a, int i) {
  int lo, hi, kv;
  raw_seq(a, i, lo, hi, kv);
  return make_seq(a, lo, hi, kv, i < a.groups);
}

// Whether a packed token belongs to a sequence (rows behind the last one are left alone).
__device__ __forceinline__ bool token_owned(const PagedArgs& a, long long tok) {
  return tok >= a.cu_seqlens[0] && tok < a.cu_seqlens[a.N];
}
// Whether it belongs to a group (of a call with groups).
__device__ __forceinline__ bool token_grouped(const PagedArgs& a, long long tok) {
  const int g0 = min(max(a.cu_groups[0], 0), a.N), g1 = min(max(a.cu_groups[a.groups], 0), a.N);
  return tok >= a.cu_seqlens[g0] && tok < a.cu_seqlens[g1];
}

// The query at position `pos` sees `key`: causal, and with a window the last `window` keys
// and the first `sinks` ones.
__device__ __forceinline__ bool visible(const PagedArgs& a, int pos, int key) {
  return key <= pos && (a.window == 0 || key > pos - a.window || key < a.sinks);
}

// Keys that any of the tokens t0..t1 of a sequence sees: [0, sinks) and [lo, hi).
struct KeyRange {
  int sinks, lo, hi;
};

__device__ __forceinline__ KeyRange key_range(const PagedArgs& a, const Seq& s, int t0, int t1) {
  KeyRange r;
  r.hi = max(min(s.kv, s.pos0 + t1 + 1), 0);
  r.lo = a.window ? max(0, max(s.pos0 + t0, 0) - a.window + 1) : 0;
  r.lo = min(r.lo, r.hi);
  r.sinks = min(a.window ? a.sinks : 0, r.lo);
  return r;
}

// The v-th key of a range.
__device__ __forceinline__ int virtual_key(const KeyRange& r, int v) {
  return v < r.sinks ? v : v - r.sinks + r.lo;
}

// The page that holds `key`, clamped into the cache: a bad table entry gives wrong numbers
// but no access outside it.
__device__ __forceinline__ int page_of(const PagedArgs& a, int n, int key) {
  const int p = __ldg(table_of(a, n) + key / a.page_size);
  return min(max(p, 0), a.num_pages - 1);
}

// Row (of D elements) of a key in the cache [num_pages, Hkv, page_size, D].
__device__ __forceinline__ long long cache_row(const PagedArgs& a, int n, int hkv, int key) {
  return ((long long)page_of(a, n, key) * a.Hkv + hkv) * a.page_size + key % a.page_size;
}

// The list and row tile behind a block's number, tiles of `rows` query rows counted over
// the lists in order.  All NT threads call; false when there is no such tile.
template <int NT>
__device__ bool find_row_tile(const PagedArgs& a, int rows, int number, int* s2, int& seq,
                              int& tile) {
  __shared__ int s_warp[NT / 32];
  const int G = a.Hq / a.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int before = 0;  // tiles of the sequences before this round
  for (int base = 0; base < lists(a); base += NT) {
    const int n = base + tid;
    int t = 0;
    if (n < lists(a)) {
      int lo, hi, kv;
      raw_seq(a, n, lo, hi, kv);
      lo = min(max(lo, 0), a.total_T);
      hi = min(max(hi, lo), a.total_T);
      t = (int)(((long long)(hi - lo) * G + rows - 1) / rows);
    }
    int sum = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) s_warp[warp] = sum;
    if (tid == 0) s2[0] = -1;
    __syncthreads();
    int all = 0, pre = before;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) pre += s_warp[w];
      all += s_warp[w];
    }
    pre += sum - t;
    if (number >= pre && number < pre + t) {
      s2[0] = n;
      s2[1] = number - pre;
    }
    __syncthreads();
    if (s2[0] >= 0) {
      seq = s2[0];
      tile = s2[1];
      return true;
    }
    before += all;
    __syncthreads();
  }
  return false;
}

}  // namespace kda
