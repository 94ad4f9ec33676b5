// cache.cu -- the paged cache held in 4 bits: appending a batch's keys (rotated on the way) and
// values, and reading rows back as the values that they stand for.
//
// Both kernels are bound by HBM for prompts (every element read once, 4.5 bits of a cached one
// written or read) and by latency for single tokens.  A thread owns one token and eight
// neighbouring channels: eight codes are one 32-bit word of the cache, the 64 channels of a
// (step, lo) pair are eight neighbouring lanes, so that a group's range costs three shuffles
// and nothing goes through shared memory.  The thread finds its sequence, page and angles once
// and walks the heads (keys, values and queries numbered through); few tokens spread the heads
// over more blocks.
#include <cuda_fp16.h>

#include <cmath>

#include "cache.cuh"
#include "common.h"
#include "launch.h"
#include "rope.cuh"
#include "serving.h"

namespace ra {
namespace {

constexpr int kThreads = 128;

struct RowPtr {
  const void* in;
  void* out;
  int64_t in_n, in_h, out_n, out_h;  // strides of token and head (elements)
  int vec;                           // 16-byte accesses fit
};

struct AppendArgs {
  CacheDims c;
  uint8_t* cache;
  const int *table, *indptr, *kv_len;
  const double* freqs;
  double amplitude;
  int r, half;
  RowPtr k, v, q;  // q.in null: no queries
  int heads_per_chunk;
  uint32_t* err;
};

struct ReadArgs {
  CacheDims c;
  const uint8_t* cache;
  const int *table, *indptr, *kv_len;
  RowPtr k, v;  // out null: not wanted
  int heads_per_chunk;
  uint32_t* err;
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, bool vec, float (&f)[8]) {
  if (vec) {
    if constexpr (sizeof(T) == 2) {
      Vec<T, 8> v;
      v.load(p);
      v.get(f);
    } else {
      const float4 a = reinterpret_cast<const float4*>(p)[0];
      const float4 b = reinterpret_cast<const float4*>(p)[1];
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
      f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      Vec<T, 1> v;
      float g[1];
      v.load(p + j);
      v.get(g);
      f[j] = g[0];
    }
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, bool vec, const float (&f)[8]) {
  if (vec) {
    if constexpr (sizeof(T) == 2) {
      Vec<T, 8> v;
      v.set(f);
      v.store(p);
    } else {
      reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      Vec<T, 1> v;
      const float g[1] = {f[j]};
      v.set(g);
      v.store(p + j);
    }
  }
}

// The sequence whose rows hold token t: the largest b with indptr[b] <= t, by a 32-ary search
// of the whole (converged) warp; t is the same in every lane.
__device__ __forceinline__ int find_sequence(const int* __restrict__ indptr, int B, int t) {
  int lo = 0, hi = B;
  const int lane = threadIdx.x % 32;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const int below = __popc(__ballot_sync(0xffffffffu, at < hi && indptr[at] <= t));
    lo += (below > 0 ? below - 1 : 0) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Where token t of the batch lives: its position, or -1 if it belongs to no sequence or to a
// faulty one (recorded).  The whole warp calls this with the tokens of its lane groups.
template <int LANES>
__device__ __forceinline__ int locate(const CacheDims& c, const int* indptr, const int* kv_len,
                                      int t, uint32_t* err, int kid, int& seq) {
  const int lane = threadIdx.x % 32;
  seq = -1;
#pragma unroll
  for (int g = 0; g < 32 / LANES; ++g) {
    const int tg = __shfl_sync(0xffffffffu, t, g * LANES);
    const int b = find_sequence(indptr, c.B, tg);
    if (lane / LANES == g) seq = b;
  }
  if (t >= c.T) return -1;
  const int q0 = indptr[seq], q1 = indptr[seq + 1], L = kv_len[seq];
  int fault = sequence_fault(c, q0, q1, L);
  if (!fault && (t < q0 || t >= q1)) return -1;  // before the first or behind the last sequence
  if (!fault && L < q1 - q0) fault = RA_CACHE_BAD_LENGTH;
  if (fault) {
    record_cache_fault(err, kid, fault, seq);
    return -1;
  }
  return L - (q1 - q0) + (t - q0);
}

// The first block looks over every sequence, so that a fault is reported even where no token
// of this launch meets it.
__device__ __forceinline__ void check_batch(const CacheDims& c, const int* indptr,
                                            const int* kv_len, uint32_t* err, int kid) {
  if (blockIdx.x != 0 || blockIdx.y != 0) return;
  for (int b = threadIdx.x; b < c.B; b += blockDim.x) {
    const int q0 = indptr[b], q1 = indptr[b + 1], L = kv_len[b];
    int fault = sequence_fault(c, q0, q1, L);
    if (!fault && L < q1 - q0) fault = RA_CACHE_BAD_LENGTH;
    if (fault) record_cache_fault(err, kid, fault, b);
  }
}

// Eight channels of a group of 64 (eight neighbouring lanes) to codes, and the group's pair.
// The roundings are those of the documented definition, one by one.
__device__ __forceinline__ uint32_t quantise8(float (&x)[8], bool& beyond, __half2& pair) {
  float lo = INFINITY, hi = -INFINITY;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (!(fabsf(x[j]) <= RA_CACHE_LIMIT)) {
      beyond = true;
      x[j] = isnan(x[j]) ? 0.f : copysignf(RA_CACHE_LIMIT, x[j]);
    }
    lo = fminf(lo, x[j]);
    hi = fmaxf(hi, x[j]);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const __half lo16 = __float2half_rn(lo);
  const float base = __half2float(lo16);
  const __half step16 = __float2half_rn(fmaxf(__fmul_rn(__fsub_rn(hi, base), 1.f / 15.f), 0.f));
  const float step = __half2float(step16);
  const float inv = step > 0.f ? __fdiv_rn(1.f, step) : 0.f;
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float code = rintf(__fmul_rn(__fsub_rn(x[j], base), inv));
    w |= (uint32_t)fminf(fmaxf(code, 0.f), 15.f) << (4 * j);
  }
  pair = __halves2half2(step16, lo16);
  return w;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const AppendArgs a) {
  constexpr int U = D / 8;  // threads of a token
  const CacheDims& c = a.c;
  check_batch(c, a.indptr, a.kv_len, a.err, K_CACHE_APPEND);
  const int u = threadIdx.x % U, c0 = u * 8;
  const int t = blockIdx.x * (kThreads / U) + threadIdx.x / U;
  int seq;
  const int pos = locate<U>(c, a.indptr, a.kv_len, t, a.err, K_CACHE_APPEND, seq);
  const bool live = pos >= 0;
  const int page =
      live ? page_of(c, a.table, seq, pos / kBlock, a.err, K_CACHE_APPEND) : -1;
  const int blk = live ? (pos / kBlock) % c.page_blocks : 0, row = live ? pos % kBlock : 0;
  const int h_lo = blockIdx.y * a.heads_per_chunk, h_hi = h_lo + a.heads_per_chunk;

  // angles of the channel pairs (interleaved) or channels (half) that lie in the rotated part
  float2 cs[8];
  const bool turns = live && (h_lo < c.Hkv || h_hi > 2 * c.Hkv) && c0 < a.r;
  if (turns) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!a.half && j >= 4) continue;
      const int ch = a.half ? c0 + j : c0 + 2 * j;
      const int m = a.half ? (ch < a.r / 2 ? ch : ch - a.r / 2) : ch / 2;
      if (ch < a.r) cs[j] = cos_sin((double)pos, a.freqs[m], a.amplitude);
    }
  }
  // x (own channels of a row at p) rotated in place
  auto rotate = [&](const T* p, bool vec, float (&x)[8]) {
    if (c0 >= a.r) return;
    if (a.half) {
      float y[8];  // the partner channels
      const int first = c0 < a.r / 2 ? c0 + a.r / 2 : c0 - a.r / 2;
      if ((a.r / 2) % 8 == 0) {
        load8(p + first, vec, y);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int ch = c0 + j;
          y[j] = 0.f;
          if (ch < a.r) {
            Vec<T, 1> v;
            float g[1];
            v.load(p + (ch < a.r / 2 ? ch + a.r / 2 : ch - a.r / 2));
            v.get(g);
            y[j] = g[0];
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int ch = c0 + j;
        if (ch < a.r / 2)
          x[j] = turn(cs[j], x[j], y[j]).x;
        else if (ch < a.r)
          x[j] = turn(cs[j], y[j], x[j]).y;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (c0 + 2 * j >= a.r) break;
        const float2 y = turn(cs[j], x[2 * j], x[2 * j + 1]);
        x[2 * j] = y.x;
        x[2 * j + 1] = y.y;
      }
    }
  };

  bool beyond = false;
  for (int h = h_lo; h < h_hi && h < 2 * c.Hkv + (a.q.in ? c.Hq : 0); ++h) {
    if (h < 2 * c.Hkv) {
      // keys (rotated), then values: the whole warp takes part in the groups' shuffles
      const bool is_k = h < c.Hkv;
      const int hh = is_k ? h : h - c.Hkv;
      const RowPtr& p = is_k ? a.k : a.v;
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (live) {
        const T* src = static_cast<const T*>(p.in) + (int64_t)t * p.in_n + (int64_t)hh * p.in_h;
        load8(src + c0, p.vec, x);
        if (is_k) rotate(src, p.vec, x);
      }
      __half2 pair;
      const uint32_t w = quantise8(x, beyond, pair);
      if (page >= 0) {
        uint8_t* block =
            a.cache + block_at(c, page, hh, blk) + (is_k ? 0 : value_offset(D));
        *reinterpret_cast<uint32_t*>(block + row * (D / 2) + u * 4) = w;
        if (u % 8 == 0)
          *reinterpret_cast<__half2*>(block + code_bytes(D) + (row * (D / kGroup) + u / 8) * 4) =
              pair;
      }
    } else {
      const int hh = h - 2 * c.Hkv;
      float x[8];
      if (live) {
        const T* src = static_cast<const T*>(a.q.in) + (int64_t)t * a.q.in_n +
                       (int64_t)hh * a.q.in_h;
        load8(src + c0, a.q.vec, x);
        rotate(src, a.q.vec, x);
      }
      // in place, a half-layout row's partner channels are read by other lanes of the warp
      // before any lane writes its own
      __syncwarp();
      if (live)
        store8(static_cast<T*>(a.q.out) + (int64_t)t * a.q.out_n + (int64_t)hh * a.q.out_h + c0,
               a.q.vec, x);
    }
  }
  if (beyond) atomicCAS(a.err, 0u, (uint32_t)RA_ERR_RANGE);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const ReadArgs a) {
  constexpr int U = D / 8;
  const CacheDims& c = a.c;
  check_batch(c, a.indptr, a.kv_len, a.err, K_CACHE_READ);
  const int u = threadIdx.x % U, c0 = u * 8;
  const int t = blockIdx.x * (kThreads / U) + threadIdx.x / U;
  int seq;
  const int pos = locate<U>(c, a.indptr, a.kv_len, t, a.err, K_CACHE_READ, seq);
  if (pos < 0) return;
  const int page = page_of(c, a.table, seq, pos / kBlock, a.err, K_CACHE_READ);
  const int blk = (pos / kBlock) % c.page_blocks, row = pos % kBlock;
  const int h_lo = blockIdx.y * a.heads_per_chunk;
  const int h_hi = min(h_lo + a.heads_per_chunk, 2 * c.Hkv);
#pragma unroll 4
  for (int h = h_lo; h < h_hi; ++h) {
    const bool is_k = h < c.Hkv;
    const int hh = is_k ? h : h - c.Hkv;
    const RowPtr& p = is_k ? a.k : a.v;
    if (!p.out) continue;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (page >= 0) {
      const uint8_t* block = a.cache + block_at(c, page, hh, blk) + (is_k ? 0 : value_offset(D));
      const uint32_t w = *reinterpret_cast<const uint32_t*>(block + row * (D / 2) + u * 4);
      const float2 pair = __half22float2(*reinterpret_cast<const __half2*>(
          block + code_bytes(D) + (row * (D / kGroup) + u / 8) * 4));
#pragma unroll
      for (int j = 0; j < 8; ++j)  // step * code is exact in fp32: one rounding, of the sum
        x[j] = fmaf(pair.x, (float)((w >> (4 * j)) & 15u), pair.y);
    }
    store8(static_cast<T*>(p.out) + (int64_t)t * p.out_n + (int64_t)hh * p.out_h + c0, p.vec, x);
  }
}

// ------------------------------------------------------------------ host
bool aligned_to(const void* p, size_t a) {
  return p && (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// [T, H, d] rows for a cache call; written rows must not overlap.
ra_status check_token_rows(const ra_rows* r, const ra_cache& p, int64_t H, bool written) {
  if (!r || !aligned_to(r->ptr, elem_bytes(p.dtype)) || r->H != H) return RA_ERR_INVALID_ARG;
  if (r->stride_n < 0 || r->stride_h < 0 || r->stride_n > (int64_t(1) << 40) ||
      r->stride_h > (int64_t(1) << 40))
    return RA_ERR_INVALID_ARG;
  if (written) {
    const bool n_outer = r->stride_n >= r->stride_h;
    const int64_t in_s = n_outer ? r->stride_h : r->stride_n, in_e = n_outer ? H : p.T;
    const int64_t out_s = n_outer ? r->stride_n : r->stride_h, out_e = n_outer ? p.T : H;
    if (in_e > 1 && in_s < p.d) return RA_ERR_INVALID_ARG;
    const int64_t span = (in_e > 1 ? in_s * (in_e - 1) : 0) + p.d;
    if (out_e > 1 && out_s < span) return RA_ERR_INVALID_ARG;
  }
  return RA_OK;
}

int vectors_fit(const ra_rows& r, int32_t dtype) {
  const int64_t V = (int64_t)(16 / elem_bytes(dtype));
  return aligned_to(r.ptr, 16) && r.stride_n % V == 0 && r.stride_h % V == 0;
}

// Heads per block: all of them, or fewer until the launch has about eight blocks per SM.
int chunk_of(int64_t token_blocks, int64_t heads) {
  const int64_t want = (kRotaryBlocks + token_blocks - 1) / token_blocks;
  const int64_t chunks = std::max<int64_t>(1, std::min<int64_t>(want, heads));
  return (int)((heads + chunks - 1) / chunks);
}

}  // namespace

ra_status check_cache(const ra_cache* p) {
  if (!p) return RA_ERR_INVALID_ARG;
  if (p->dtype != RA_F32 && p->dtype != RA_BF16) return RA_ERR_INVALID_ARG;
  if (p->causal != 0 && p->causal != 1) return RA_ERR_INVALID_ARG;
  if (p->B < 1 || p->T < 0 || p->Hkv < 1 || p->Hq < 1 || p->pages < 1 || p->max_pages < 1 ||
      p->max_q < 0 || p->window < 0)
    return RA_ERR_INVALID_ARG;
  if (p->page_size < kBlock || p->page_size % kBlock) return RA_ERR_INVALID_ARG;
  if (!p->causal && p->window) return RA_ERR_INVALID_ARG;
  if (!(p->scale >= 0.0) || !std::isfinite((float)p->scale)) return RA_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return RA_ERR_UNSUPPORTED;
  if (p->B > 65536 || p->T > (int64_t(1) << 30) || p->Hkv > 1024 || p->Hq > 4096 ||
      p->pages > (int64_t(1) << 30) || p->page_size > 4096 || p->window > (int64_t(1) << 30) ||
      p->max_q > (int64_t(1) << 30) || p->max_pages > (int64_t(1) << 30) / p->page_size)
    return RA_ERR_UNSUPPORTED;
  if (p->T * p->Hq > (int64_t(1) << 38) / p->d) return RA_ERR_UNSUPPORTED;
  if (p->Hq % p->Hkv) return RA_ERR_INVALID_ARG;
  return RA_OK;
}

CacheDims cache_dims(const ra_cache& p) {
  CacheDims c{};
  c.B = (int)p.B, c.T = (int)p.T, c.Hq = (int)p.Hq, c.Hkv = (int)p.Hkv, c.d = (int)p.d;
  c.pages = (int)p.pages, c.page_blocks = (int)(p.page_size / kBlock);
  c.max_pages = (int)p.max_pages;
  c.max_q = (int)(p.max_q ? std::min(p.max_q, p.T) : p.T);
  c.window = (int)p.window, c.causal = p.causal;
  c.scale = p.scale != 0.0 ? (float)p.scale : (float)(1.0 / std::sqrt((double)p.d));
  return c;
}

// The arguments that every cache call shares.
ra_status check_cache_call(const ra_cache* p, const void* cache, const int32_t* table,
                           const int32_t* indptr, const int32_t* kv_len, void* ws,
                           size_t ws_bytes) {
  const ra_status st = check_cache(p);
  if (st != RA_OK) return st;
  if (!aligned_to(cache, 16) || !aligned_to(table, 4) || !aligned_to(indptr, 4) ||
      !aligned_to(kv_len, 4))
    return RA_ERR_INVALID_ARG;
  if (!aligned_to(ws, 256) || ws_bytes < rope_attn_cache_workspace_bytes(p))
    return RA_ERR_WORKSPACE;
  return RA_OK;
}

}  // namespace ra

using namespace ra;

extern "C" {

size_t rope_attn_cache_block_bytes(int64_t d) {
  return d == 64 || d == 128 ? (size_t)block_bytes((int)d) : 0;
}

size_t rope_attn_cache_bytes(const ra_cache* p) {
  if (check_cache(p) != RA_OK) return 0;
  return (size_t)p->pages * (size_t)p->Hkv * (size_t)(p->page_size / kBlock) *
         (size_t)block_bytes((int)p->d);
}

ra_status rope_attn_cache_append(const ra_cache* p, void* cache, const int32_t* table,
                                 const int32_t* indptr, const int32_t* kv_len,
                                 const ra_rotary* r, const double* freqs, const ra_rows* k,
                                 const ra_rows* v, const ra_rows* q, const ra_rows* q_out,
                                 void* ws, size_t ws_bytes, void* stream) {
  ra_status st = check_cache_call(p, cache, table, indptr, kv_len, ws, ws_bytes);
  if (st != RA_OK) return st;
  if ((st = check_rotary(r)) != RA_OK) return st;
  if (r->d != p->d || !aligned_to(freqs, 8)) return RA_ERR_INVALID_ARG;
  if (p->T == 0) return RA_OK;
  if ((st = check_token_rows(k, *p, p->Hkv, false)) != RA_OK) return st;
  if ((st = check_token_rows(v, *p, p->Hkv, false)) != RA_OK) return st;
  if ((q == nullptr) != (q_out == nullptr)) return RA_ERR_INVALID_ARG;
  if (q) {
    if ((st = check_token_rows(q, *p, p->Hq, false)) != RA_OK) return st;
    if ((st = check_token_rows(q_out, *p, p->Hq, true)) != RA_OK) return st;
    if (q->ptr == q_out->ptr && (q->stride_n != q_out->stride_n || q->stride_h != q_out->stride_h))
      return RA_ERR_INVALID_ARG;
  }
  AppendArgs a{};
  a.c = cache_dims(*p);
  a.cache = static_cast<uint8_t*>(cache);
  a.table = table, a.indptr = indptr, a.kv_len = kv_len;
  a.freqs = freqs, a.amplitude = r->amplitude, a.r = (int)r->rot_dim;
  a.half = r->layout == RA_HALF;
  a.k = {k->ptr, nullptr, k->stride_n, k->stride_h, 0, 0, vectors_fit(*k, p->dtype)};
  a.v = {v->ptr, nullptr, v->stride_n, v->stride_h, 0, 0, vectors_fit(*v, p->dtype)};
  if (q)
    a.q = {q->ptr, q_out->ptr, q->stride_n, q->stride_h, q_out->stride_n, q_out->stride_h,
           vectors_fit(*q, p->dtype) && vectors_fit(*q_out, p->dtype)};
  a.err = static_cast<uint32_t*>(ws);
  const int tokens = kThreads / (a.c.d / 8);
  const int64_t gx = (p->T + tokens - 1) / tokens;
  const int64_t heads = 2 * p->Hkv + (q ? p->Hq : 0);
  a.heads_per_chunk = chunk_of(gx, heads);
  const dim3 grid((unsigned)gx, (unsigned)((heads + a.heads_per_chunk - 1) / a.heads_per_chunk));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const TimingScope timed(K_CACHE_APPEND, s);
  if (p->dtype == RA_BF16) {
    if (p->d == 64) cache_append_kernel<__nv_bfloat16, 64><<<grid, kThreads, 0, s>>>(a);
    else cache_append_kernel<__nv_bfloat16, 128><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (p->d == 64) cache_append_kernel<float, 64><<<grid, kThreads, 0, s>>>(a);
    else cache_append_kernel<float, 128><<<grid, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? RA_OK : RA_ERR_CUDA;
}

ra_status rope_attn_cache_read(const ra_cache* p, const void* cache, const int32_t* table,
                               const int32_t* indptr, const int32_t* kv_len, const ra_rows* k,
                               const ra_rows* v, void* ws, size_t ws_bytes, void* stream) {
  ra_status st = check_cache_call(p, cache, table, indptr, kv_len, ws, ws_bytes);
  if (st != RA_OK) return st;
  if (p->T == 0) return RA_OK;
  if (k && (st = check_token_rows(k, *p, p->Hkv, true)) != RA_OK) return st;
  if (v && (st = check_token_rows(v, *p, p->Hkv, true)) != RA_OK) return st;
  if (!k && !v) return RA_OK;
  ReadArgs a{};
  a.c = cache_dims(*p);
  a.cache = static_cast<const uint8_t*>(cache);
  a.table = table, a.indptr = indptr, a.kv_len = kv_len;
  if (k) a.k = {nullptr, k->ptr, 0, 0, k->stride_n, k->stride_h, vectors_fit(*k, p->dtype)};
  if (v) a.v = {nullptr, v->ptr, 0, 0, v->stride_n, v->stride_h, vectors_fit(*v, p->dtype)};
  a.err = static_cast<uint32_t*>(ws);
  const int tokens = kThreads / (a.c.d / 8);
  const int64_t gx = (p->T + tokens - 1) / tokens;
  a.heads_per_chunk = chunk_of(gx, 2 * p->Hkv);
  const dim3 grid((unsigned)gx,
                  (unsigned)((2 * p->Hkv + a.heads_per_chunk - 1) / a.heads_per_chunk));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const TimingScope timed(K_CACHE_READ, s);
  if (p->dtype == RA_BF16) {
    if (p->d == 64) cache_read_kernel<__nv_bfloat16, 64><<<grid, kThreads, 0, s>>>(a);
    else cache_read_kernel<__nv_bfloat16, 128><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (p->d == 64) cache_read_kernel<float, 64><<<grid, kThreads, 0, s>>>(a);
    else cache_read_kernel<float, 128><<<grid, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? RA_OK : RA_ERR_CUDA;
}

}  // extern "C"
