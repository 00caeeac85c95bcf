// short_conv.hpp -- gfx950 device code of the short causal convolution over
// packed sequences, depthwise:
//
//   a[t] = bias + sum_k w[k] x[t-K+1+k],  y[t] = a or silu(a)
//
// with x before a sequence's first token from its window (or 0); of its single
// token; and of its gradients
//   da = dy act'(a),  dx[t] = sum_k w[k] da[t+K-1-k],  dw[k] = sum_t da[t] x[t-K+1+k],
// silu'(a) = s (1 + a (1 - s)), s = 1 / (1 + exp(-a)).
//
// A lane holds V neighbouring channels (4, or one where rows do not start on 4) and walks
// a tile of tokens with the last three inputs in registers; a wave covers 64 V channels,
// and the waves of a workgroup lie side by side on the same tokens.  Bound by memory: a
// tile reads K - 1 rows more than its own, and they come from memory again, since
// neighbouring tiles lie on different XCDs (32768 x 2560 bf16, tiles of 16: 202 MB read
// for 168 MB of x; neighbours on one XCD gained nothing).  Loads and stores go
// through the caches: loads past them gain 1% in a forward pass and lose 9% where the
// gradients follow it (16384 x 1536 fp32 114 -> 124 us); stores past them change nothing.
#pragma once

#include "add_norm.hpp"
#include "packed.hpp"

namespace ssmc {

using ssma::load_v;
using ssma::Raw;
using ssma::store_v;
using ssmn::bf16_t;
using ssmn::sigmoid;
using ssmq::Seqs;
using ssmq::seq_resumed;
using ssmq::seq_slot;
using ssmq::seq_start;
using ssmq::seqs_before;

constexpr int kAhead = 4;      // rows requested before the current ones are used

struct ConvParams {
  const void* x;
  const float* w;        // (C, K)
  const float* b;        // or null
  float* state;          // (slots, C, K - 1) or null
  void* y;               // backward: dx
  const void* dy;
  float* part;           // backward: (tiles, C (K + 1)): sums for dweight, then dbias; or null
  int64_t C, xs, ds;     // row strides of x and dy
  Seqs q;
  int32_t tile, tiles, cgroups;
  int32_t silu;
};

// N floats at p: by 16 bytes where a lane holds several channels.
template <int N, int V>
__device__ __forceinline__ void load_n(float* v, const float* p) {
  if constexpr (V == 1) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = p[j];
  } else {
    load_v<N>(v, p);
  }
}

// A lane's taps, oldest first, and bias.  (The taps of a channel, and the channels
// of a lane, lie side by side.)
template <int V, int K>
struct Filter {
  float w[K][V], b[V];
  __device__ __forceinline__ void load(const ConvParams& p, int64_t c) {
    float v[V * K];
    load_n<V * K, V>(v, p.w + c * K);
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int k = 0; k < K; ++k) w[k][i] = v[i * K + k];
      b[i] = 0.0f;
    }
    if (p.b) load_v<V>(b, p.b + c);
  }
};

// The last inputs: [k] the one k + 1 tokens back.
template <int V, int K>
struct Past {
  static constexpr int B = K > 1 ? K - 1 : 1;
  float v[B][V];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < B; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = 0.0f;
  }
  __device__ __forceinline__ void push(const float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int k = B - 1; k > 0; --k) v[k][i] = v[k - 1][i];
      v[0][i] = x[i];
    }
  }
};

// The convolution at one token, from the newest tap on.
template <int V, int K>
__device__ __forceinline__ void taps_sum(const Filter<V, K>& f, const float (&x)[V], const Past<V, K>& h,
                                         float (&a)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float v = fmaf(f.w[K - 1][i], x[i], f.b[i]);
#pragma unroll
    for (int k = 1; k < K; ++k) v = fmaf(f.w[K - 1 - k][i], h.v[k - 1][i], v);
    a[i] = v;
  }
}

// A window in memory is (channels, K - 1), oldest input first.  A lane's V (K - 1)
// floats lie side by side.
template <int V, int K>
__device__ __forceinline__ void load_window(Past<V, K>& h, const float* p) {
  if constexpr (K > 1) {
    float v[V * (K - 1)];
    load_n<V * (K - 1), V>(v, p);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < K - 1; ++j) h.v[K - 2 - j][i] = v[i * (K - 1) + j];
  }
}
template <int V, int K>
__device__ __forceinline__ void store_window(const Past<V, K>& h, float* p) {
  if constexpr (K > 1) {
    float v[V * (K - 1)];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < K - 1; ++j) v[i * (K - 1) + j] = h.v[K - 2 - j][i];
    if constexpr (V == 1) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) p[j] = v[j];
    } else {
      store_v<V * (K - 1)>(p, v);
    }
  }
}

// Where a tile that nominally begins at token b begins.  A sequence's window is
// read, and moved on in place, by the one tile that holds its first token: that
// tile also takes the tokens behind it whose taps reach into the window.
template <int K>
__device__ __forceinline__ int32_t tile_edge(const ConvParams& p, int32_t b) {
  if (!p.state || K < 3 || b <= 0 || b >= p.q.tokens) return b;
  const int32_t i = seqs_before(p.q, b) - 1;
  if (i < 0) return b;
  const int32_t first = seq_start(p.q, i), end = seq_start(p.q, i + 1);
  if (end <= b || b - first >= K - 1) return b;
  return first + K - 1 < end ? first + K - 1 : end;
}

template <typename T, int V, int K>
__global__ __launch_bounds__(256) void k_short_conv(ConvParams p) {
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int64_t id = int64_t(blockIdx.x) * 4 + wave;
  const int32_t tile = int32_t(id / p.cgroups);
  if (tile >= p.tiles) return;
  const int64_t c = (id % p.cgroups * 64 + (threadIdx.x & 63)) * V;
  const bool live = c < p.C;
  const int32_t n0 = tile * p.tile, n1 = p.q.tokens - n0 > p.tile ? n0 + p.tile : p.q.tokens;
  const int32_t t0 = tile_edge<K>(p, n0), t1 = tile_edge<K>(p, n1);
  const int32_t lo = seq_start(p.q, 0), hi = seq_start(p.q, p.q.S);
  const int32_t from = t0 > lo ? t0 : lo, to = t1 < hi ? t1 : hi;
  const T* x = static_cast<const T*>(p.x) + c;
  T* y = static_cast<T*>(p.y) + c;
  Filter<V, K> f;
  if (live) f.load(p, c);
  Past<V, K> h;
  h.clear();

  // A sequence's beginning: its window into h, and the window behind its last token
  // to its slot.
  auto begin = [&](int32_t s, int32_t first, int32_t end) {
    const int32_t slot = p.state ? seq_slot(p.q, s) : -1;
    h.clear();
    if (K == 1 || slot < 0 || !live) return;
    float* win = p.state + (int64_t(slot) * p.C + c) * (K - 1);
    if (seq_resumed(p.q, s)) load_window<V, K>(h, win);
    Past<V, K> moved;
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      // the input k + 1 tokens before the end
      const int32_t t = end - 1 - k;
      if (t >= first) {
        load_v<V>(moved.v[k], x + int64_t(t) * p.xs);
      } else {
        // of the old window: first - 1 - t tokens further back than its newest
#pragma unroll
        for (int m = 0; m < K - 1; ++m)
          if (first - 1 - t == m) {
#pragma unroll
            for (int i = 0; i < V; ++i) moved.v[k][i] = h.v[m][i];
          }
      }
    }
    store_window<V, K>(moved, win);
  };

  int32_t s = seqs_before(p.q, from);
  if (s > 0 && from < to && seq_start(p.q, s) > from) {
    // within a sequence: the inputs before the tile (with a state all of them are the sequence's own)
    const int32_t first = seq_start(p.q, s - 1);
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
      if (live && from - 1 - k >= first) load_v<V>(h.v[k], x + int64_t(from - 1 - k) * p.xs);
  }
  int32_t next = s < p.q.S ? seq_start(p.q, s) : INT32_MAX;
  // the sequences that begin at token t, the empty ones before the one that holds it
  auto meet = [&](int32_t t) {
    while (next <= t) {
      const int32_t end = seq_start(p.q, s + 1);
      begin(s, next, end > next ? end : next);
      ++s;
      next = s < p.q.S ? seq_start(p.q, s) : INT32_MAX;
    }
  };

  Raw<T, V> cur[kAhead], nxt[kAhead];
  auto rows = [&](Raw<T, V> (&v)[kAhead], int32_t t) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (live && t + j < to) v[j].template load<true>(x + int64_t(t + j) * p.xs);
  };
  if (from < to) rows(cur, from);
  for (int32_t t = from; t < to; t += kAhead) {
    rows(nxt, t + kAhead);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (t + j >= to) break;
      if (next <= t + j) meet(t + j);
      float u[V], a[V];
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] = cur[j].at(i);
      taps_sum<V, K>(f, u, h, a);
      if (p.silu) {
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] *= sigmoid(a[i]);
      }
      if (live) store_v<V>(y + int64_t(t + j) * p.C, a);
      h.push(u);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) cur[j] = nxt[j];
  }
  // empty sequences behind the last token: of the tile whose range holds their place
  const int32_t at = from > to ? from : to;
  if (at < t1 || t1 == p.q.tokens) meet(at);
}

// One token of every row of the batch: a lane to V channels of kStepRows neighbouring
// rows, which share its taps.  Bound by memory, the windows above all.
constexpr int kStepRows = 2;

template <typename T, int V, int K>
__global__ __launch_bounds__(256) void k_short_conv_step(ConvParams p) {
  const int64_t c = (int64_t(blockIdx.x) * 256 + threadIdx.x) * V;
  if (c >= p.C) return;
  Filter<V, K> f;
  f.load(p, c);
  for (int64_t row0 = int64_t(blockIdx.y) * kStepRows; row0 < p.q.S; row0 += int64_t(gridDim.y) * kStepRows) {
    // all rows are read before any is written
    float x[kStepRows][V];
    Past<V, K> h[kStepRows];
    float* win[kStepRows];
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
      const int64_t row = row0 + r < p.q.S ? row0 + r : p.q.S - 1;
      const int32_t slot = p.q.slot ? ((ssmq::const_i32_ptr)(p.q.slot))[row] : int32_t(row);
      win[r] = K > 1 && slot >= 0 && slot < p.q.slots ? p.state + (int64_t(slot) * p.C + c) * (K - 1) : nullptr;
      h[r].clear();
      if (win[r]) load_window<V, K>(h[r], win[r]);
      load_v<V>(x[r], static_cast<const T*>(p.x) + row * p.xs + c);
    }
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
      if (row0 + r >= p.q.S) break;
      float a[V];
      taps_sum<V, K>(f, x[r], h[r], a);
      if (p.silu) {
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] *= sigmoid(a[i]);
      }
      store_v<V>(static_cast<T*>(p.y) + (row0 + r) * p.C + c, a);
      h[r].push(x[r]);
      if (win[r]) store_window<V, K>(h[r], win[r]);
    }
  }
}

// Gradients: a tile walks its tokens and the K - 1 behind them, whose da reach back
// into it; dx of a token leaves when the da of the last of those after it, or the end
// of its sequence, is known.
template <typename T, int V, int K>
__global__ __launch_bounds__(256) void k_short_conv_bwd(ConvParams p) {
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int64_t id = int64_t(blockIdx.x) * 4 + wave;
  const int32_t tile = int32_t(id / p.cgroups);
  if (tile >= p.tiles) return;
  const int64_t c = (id % p.cgroups * 64 + (threadIdx.x & 63)) * V;
  const bool live = c < p.C;
  const int32_t t0 = tile * p.tile, t1 = p.q.tokens - t0 > p.tile ? t0 + p.tile : p.q.tokens;
  const int32_t lo = seq_start(p.q, 0), hi = seq_start(p.q, p.q.S);
  const int32_t from = t0 > lo ? t0 : lo;
  int32_t to = hi - t1 > K - 1 ? t1 + K - 1 : hi;   // tokens whose da are formed
  const T* x = static_cast<const T*>(p.x) + c;
  const T* dy = static_cast<const T*>(p.dy) + c;
  T* dx = static_cast<T*>(p.y) + c;
  Filter<V, K> f;
  Past<V, K> h, d;   // inputs, and da, of the last tokens
  float dw[K][V], db[V];
  if (live) f.load(p, c);
  h.clear();
  d.clear();
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int k = 0; k < K; ++k) dw[k][i] = 0.0f;
    db[i] = 0.0f;
  }

  // tokens of no sequence
  const float none[V] = {};
  if (live) {
    for (int32_t t = t0; t < t1 && t < lo; ++t) store_v<V>(dx + int64_t(t) * p.C, none);
    for (int32_t t = t0 > hi ? t0 : hi; t < t1; ++t) store_v<V>(dx + int64_t(t) * p.C, none);
  }
  if (from >= t1 || from >= to) {
    to = from;
  }
  int32_t s = seqs_before(p.q, from), first = from;
  if (s > 0 && from < to && seq_start(p.q, s) > from) {
    first = seq_start(p.q, s - 1);
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
      if (live && from - 1 - k >= first) load_v<V>(h.v[k], x + int64_t(from - 1 - k) * p.xs);
  }
  if (first < from) first = from;   // from here on: the first token whose dx is this walk's
  int32_t next = s < p.q.S ? seq_start(p.q, s) : INT32_MAX;

  auto put = [&](int32_t t, const float (&v)[V]) {
    if (live && t >= first && t < t1) store_v<V>(dx + int64_t(t) * p.C, v);
  };
  // dx of the tokens before t that wait for da of tokens their sequence does not have
  auto flush = [&](int32_t t) {
#pragma unroll
    for (int m = K - 1; m >= 1; --m) {
      float v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < m; ++j) v[i] += f.w[K - 1 - j][i] * d.v[m - 1 - j][i];
      }
      put(t - m, v);
    }
  };

  Raw<T, V> cx[kAhead], cd[kAhead], nx[kAhead], nd[kAhead];
  auto rows = [&](Raw<T, V> (&u)[kAhead], Raw<T, V> (&v)[kAhead], int32_t t) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (live && t + j < to) {
        u[j].template load<true>(x + int64_t(t + j) * p.xs);
        v[j].template load<true>(dy + int64_t(t + j) * p.ds);
      }
  };
  rows(cx, cd, from);
  int32_t done = from;   // tokens before it are walked
  for (int32_t t = from; t < to; t += kAhead) {
    rows(nx, nd, t + kAhead);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (t + j >= to) break;
      if (next <= t + j) {
        // a sequence begins: the one before it is complete
        flush(t + j);
        h.clear();
        d.clear();
        first = t + j;
        while (next <= t + j) {
          ++s;
          next = s < p.q.S ? seq_start(p.q, s) : INT32_MAX;
        }
        if (first >= t1) to = first;   // nothing of this tile is left
        if (t + j >= to) break;
      }
      float u[V], a[V], da[V];
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] = cx[j].at(i);
      taps_sum<V, K>(f, u, h, a);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float g = sigmoid(a[i]), dy_ = cd[j].at(i);
        da[i] = p.silu ? dy_ * (g * (1.0f + a[i] * (1.0f - g))) : dy_;
      }
      if (t + j < t1) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          dw[K - 1][i] += da[i] * u[i];
#pragma unroll
          for (int k = 1; k < K; ++k) dw[K - 1 - k][i] += da[i] * h.v[k - 1][i];
          db[i] += da[i];
        }
      }
      float v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[i] = f.w[0][i] * da[i];
#pragma unroll
        for (int k = 1; k < K; ++k) v[i] += f.w[k][i] * d.v[k - 1][i];
      }
      put(t + j - (K - 1), v);
      h.push(u);
      d.push(da);
      done = t + j + 1;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      cx[j] = nx[j];
      cd[j] = nd[j];
    }
  }
  // the walk ended with the last sequence (or behind the tile, where nothing waits)
  if (done > from && done >= first) flush(done);
  if (p.part && live) {
    float* out = p.part + int64_t(tile) * p.C * (K + 1);
    float v[V * K];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < K; ++k) v[i * K + k] = dw[k][i];
    if constexpr (V == 1) {
#pragma unroll
      for (int k = 0; k < K; ++k) out[c * K + k] = v[k];
    } else {
      store_v<V * K>(out + c * K, v);
    }
    store_v<V>(out + p.C * K + c, db);
  }
}

// The tiles' sums into dweight (C, K) and dbias (C), in order: 16 lanes of a
// workgroup share a column, each with every 16th tile, and join in LDS.
struct ConvSumParams {
  const float* part;     // (tiles, C (K + 1))
  float* dw;             // or null
  float* db;             // or null
  int64_t tiles, C, K;
};

static __global__ __launch_bounds__(256) void k_conv_sums(ConvSumParams p) {
  __shared__ float part[16][17];
  const int col = threadIdx.x & 15, lane = threadIdx.x >> 4;
  const int64_t i = int64_t(blockIdx.x) * 16 + col, n = p.C * (p.K + 1);
  float s = 0.0f;
  if (i < n) {
    int64_t k = lane;
    for (; k + 48 < p.tiles; k += 64) {
      float a[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) a[u] = p.part[(k + 16 * u) * n + i];
#pragma unroll
      for (int u = 0; u < 4; ++u) s += a[u];
    }
    for (; k < p.tiles; k += 16) s += p.part[k * n + i];
  }
  part[lane][col] = s;
  __syncthreads();
  if (lane == 0 && i < n) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) t += part[k][col];
    if (i < p.C * p.K) {
      if (p.dw) p.dw[i] = t;
    } else if (p.db) {
      p.db[i - p.C * p.K] = t;
    }
  }
}

}  // namespace ssmc
