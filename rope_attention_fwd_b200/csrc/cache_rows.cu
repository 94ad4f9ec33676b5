// cache_rows.cu -- bf16 attention over the paged 4-bit cache for a few rows per sequence and kv
// head (single tokens of grouped heads, a few tokens at once): the decode kernel.
//
// The floor is the cache itself, read once: 2 (d/2 + 4 d/64) bytes a token and kv head.  Between
// HBM and the tensor cores stands the unpacking of the codes, so the design spends as few
// instructions per code as it can and none on moving data between threads:
//
//   * Warps run on their own: each takes 32 tokens (two blocks) of a step of 128, copies its
//     blocks into a private ring of shared memory (one cp.async.bulk per block, its own
//     mbarriers) and keeps its own online softmax.  The four warps of a block meet only at the
//     end of an item.
//   * S^T = K Q^T with mma.sync.m16n8k16: 16 keys are the M rows, the (up to 8 per tile) query
//     rows the N columns.  A code c becomes the bf16 value 128 + c by or-ing it under that
//     exponent: one shift and one three-input logic operation per two codes, and the products
//     with the bf16 queries are exact.  The pair of a key and group comes in afterwards, on the
//     accumulators: s = step acc + (lo - 128 step) sum(q), 4 FMAs per 128 codes instead of one
//     per two.
//   * P V as O^T = V^T P^T: channels are the M rows, so that P^T is the B operand; movmatrix
//     turns the fp16 score tile around in registers.  Codes of two keys are interleaved with
//     one permute and become fp16 1024 + c the same way; subtracting 1024 and one packed FMA
//     give lo + step c, rounded once to fp16 (11 bits: the scores' weights P are fp16 too).
//   * Which key or channel sits in which MMA row is free as long as both products agree; it is
//     chosen so that every shared-memory read is a conflict-free or two-way 4- or 8-byte
//     access of the cache's plain channel order.
//
// mma.sync rather than tcgen05: with at most 16 query rows the tensor work is a fraction of
// what mma.sync sustains, and its operands come straight from registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "cache_attn.h"
#include "cache_sched.cuh"
#include "common.h"
#include "launch.h"
#include "sm100.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kStages = 2;             // ring of a warp, in its 32-token shares of a step
constexpr float kTau = 8.0f;           // lazy rescale of the running max, log2 units

template <int D, int NT>
struct RowsCfg {
  static constexpr int CTAS = NT == 1 ? 4 : 3;              // per SM
  static constexpr int BLOCK_BYTES = block_bytes(D);
  static constexpr int STAGE = 2 * BLOCK_BYTES;
  static constexpr int RING = kStages * STAGE;              // per warp
  static constexpr int NACC = NT * (D / 16) * 4;            // O accumulators of a lane
  static constexpr int OFF_MERGE = kWarps * RING;
  static constexpr int OFF_ML = OFF_MERGE + kWarps * 32 * NACC * 4;
  static constexpr int OFF_BAR = OFF_ML + kWarps * NT * 8 * 2 * 4;
  static constexpr int OFF_SCRATCH = OFF_BAR + kWarps * kStages * 8;
  static constexpr int SMEM = OFF_SCRATCH + 8 * (kWarps + 4);
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The 8 x 8 matrix of 16-bit elements held by the warp (lane: row lane / 4, columns
// 2 (lane % 4), + 1) transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// (x & mask) | bits in one logic operation.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(mask), "r"(bits));
  return y;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

// Codes of four channels of two keys -> their values in fp16, (key a, key b) pairs:
// x holds the four nibbles of key a in its low and of key b in its high half.
__device__ __forceinline__ void values4(uint32_t x, __half2 step, __half2 lo, uint32_t* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 c = as_half2(and_or(x >> (4 * i), 0x000f000fu, 0x64006400u));
    v[i] = as_u32(__hfma2(__hsub2(c, as_half2(0x64006400u)), step, lo));
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, RowsCfg<D, NT>::CTAS)
    cache_attn_rows_kernel(const AttnArgs a) {
  using C = RowsCfg<D, NT>;
  constexpr int NG = D / kGroup;     // groups of a row
  constexpr int TILE = 8 * NT;       // query rows
  constexpr int MT = D / 16;         // M tiles of the value product
  extern __shared__ __align__(128) uint8_t smem[];
  const CacheDims& c = a.c;
  const int G = c.Hq / c.Hkv;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r = lane / 4, t = lane % 4;
  uint8_t* ring = smem + warp * C::RING;
  const uint32_t ring_s = smem_u32(ring);
  float* merge = reinterpret_cast<float*>(smem + C::OFF_MERGE);
  float* ml_s = reinterpret_cast<float*>(smem + C::OFF_ML);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * kStages;
  const float scale_log2 = c.scale * 1.4426950408889634f;

  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&bar[i], 1);
    fence_barrier_init();
  }
  __syncwarp();
  const Run run = find_run(a, reinterpret_cast<long long*>(smem + C::OFF_SCRATCH), K_CACHE_ATTN);
  Walk<WorkOf> walk(WorkOf{a}, run, c.B);
  Segment s;
  int followers = 0, fb = 0, fh = 0, ft = 0;
  uint32_t issued = 0, consumed = 0;  // shares of this warp so far: stage = n % kStages
  int gave_up = 0;                    // a bounded wait expired: no more copies, no more waits

  // the key row of MMA row r (and r + 8: 8 keys on), chosen so that the value product's lane t
  // owns keys t, t + 4, t + 8, t + 12
  const int krow = (r & 1) * 4 + (r >> 1);

  while (walk.next(s)) {
    const long long row0 = (long long)s.tile * TILE;
    const int rows = (int)min((long long)TILE, (long long)s.w.qn * G - row0);
    // keys that the lane's query columns (8 nt + 2 t, + 1) see; the tile's first and last rows
    // bound those of all (both ends rise with the row)
    int q_lo[NT][2], q_hi[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int n = 8 * nt + 2 * t + e;
        const KeyRange k = n < rows ? row_keys(c, s.w, row0 + n, G) : KeyRange{0, 0};
        q_lo[nt][e] = k.lo;
        q_hi[nt][e] = k.hi;
      }
    const KeyRange kf = row_keys(c, s.w, row0, G), kl = row_keys(c, s.w, row0 + rows - 1, G);
    // this warp's shares of the segment's steps that hold a visible key: [i0, i1)
    const int base = s.key0 + warp * 32;   // key of share 0
    int i0 = s.s0, i1 = s.s1;
    if (kl.hi <= base) i1 = i0;
    else i1 = min(i1, (kl.hi - base + kStep - 1) / kStep);
    if (kf.lo >= base + 32) i0 = max(i0, (kf.lo - base - 32) / kStep + 1);

    // pages of the two blocks of 16 shares from `pg_base`: lane l holds block l % 2 of share
    // pg_base + l / 2; -1 behind the last token or where the table is bad
    int pg = -1, pg_base = i0 - 64;
    uint32_t present = 0;  // bits 2 stage + block: the stage's block was copied
    auto issue = [&](int i) {
      if (i - pg_base >= 16) {
        pg_base = i;
        const int key = base + (i + lane / 2) * kStep + (lane % 2) * kBlock;
        pg = -1;
        if (i + lane / 2 < i1 && key < s.w.L)
          pg = page_of(c, a.table, s.b, key / kBlock, a.err, K_CACHE_ATTN);
      }
      const int stage = issued % kStages;
      ++issued;
      uint32_t have = 0;
      int page[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        page[k] = __shfl_sync(0xffffffffu, pg, 2 * (i - pg_base) + k);
        have |= page[k] >= 0 ? 1u << k : 0u;
      }
      present = (present & ~(3u << (2 * stage))) | have << (2 * stage);
      if (lane == 0) {
        mbar_arrive_expect_tx(&bar[stage], __popc(have) * C::BLOCK_BYTES);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (page[k] >= 0) {
            const int blk = (base + i * kStep) / kBlock + k;
            bulk_load(ring + stage * C::STAGE + k * C::BLOCK_BYTES,
                      a.cache + block_at(c, page[k], s.h, blk % c.page_blocks), C::BLOCK_BYTES,
                      &bar[stage]);
          }
      }
    };
    int next = i0;
    for (; next < i1 && next < i0 + kStages && !gave_up; ++next) issue(next);

    // queries as B operands (row n = 8 nt + lane / 4): the channel pairs (i, i + 4) of each
    // eight, as the codes are unpacked; and their sums over each group
    uint32_t qb[NT][NG][8];
    float qs[NT][NG][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int n = 8 * nt + r;
      const long long row = row0 + n;
      const __nv_bfloat16* src =
          static_cast<const __nv_bfloat16*>(a.q) + (s.w.q0 + row / G) * a.q_n +
          ((long long)s.h * G + row % G) * a.q_h;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t w[4] = {0u, 0u, 0u, 0u};
          if (n < rows) {
            const __nv_bfloat16* p = src + g * kGroup + 16 * t + 8 * j;
            if (a.q_vec) {
              const uint4 v = *reinterpret_cast<const uint4*>(p);
              w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
            } else {
              const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
              for (int e = 0; e < 4; ++e) w[e] = h[2 * e] | ((uint32_t)h[2 * e + 1] << 16);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sum += __uint_as_float(w[e] << 16) + __uint_as_float(w[e] & 0xffff0000u);
          qb[nt][g][4 * j + 0] = __byte_perm(w[0], w[2], 0x5410);
          qb[nt][g][4 * j + 1] = __byte_perm(w[0], w[2], 0x7632);
          qb[nt][g][4 * j + 2] = __byte_perm(w[1], w[3], 0x5410);
          qb[nt][g][4 * j + 3] = __byte_perm(w[1], w[3], 0x7632);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        qs[nt][g][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
        qs[nt][g][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
      }
    }

    float m[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) m[nt][e] = -CUDART_INF_F, l[nt][e] = 0.f;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
    }

    for (int i = i0; i < i1; ++i) {
      if (gave_up) break;
      const int stage = consumed % kStages;
      if (!mbar_wait_warp(&bar[stage], (consumed / kStages) & 1, &gave_up, a.err, K_CACHE_ATTN, 1,
                          a.wait_ns)) {
        gave_up = 1;
        break;
      }
      ++consumed;
      const uint32_t have = present >> (2 * stage);
      const uint32_t st = ring_s + stage * C::STAGE;
      const int k0 = base + i * kStep;
      // ---- scores, log2 units: rows krow, krow + 8 of each block; columns 2t, 2t + 1
      float sc[2][NT][4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[k][nt][e] = 0.f;
        if (!(have >> k & 1)) continue;
        const uint32_t kb = st + k * C::BLOCK_BYTES;
        const uint32_t pairs = kb + code_bytes(D);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint2 wa = lds64(kb + krow * (D / 2) + g * 32 + t * 8);
          const uint2 wb = lds64(kb + (krow + 8) * (D / 2) + g * 32 + t * 8);
          const float2 pa =
              __half22float2(as_half2(lds32(pairs + (krow * NG + g) * 4)));
          const float2 pb =
              __half22float2(as_half2(lds32(pairs + ((krow + 8) * NG + g) * 4)));
          float acc[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t xa = j < 2 ? wa.x : wa.y, xb = j < 2 ? wb.x : wb.y;
            const int sh = 8 * (j % 2);
            const uint32_t a0 = and_or(xa >> sh, 0x000f000fu, 0x43004300u);
            const uint32_t a1 = and_or(xb >> sh, 0x000f000fu, 0x43004300u);
            const uint32_t a2 = and_or(xa >> (sh + 4), 0x000f000fu, 0x43004300u);
            const uint32_t a3 = and_or(xb >> (sh + 4), 0x000f000fu, 0x43004300u);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_bf16(acc[nt], a0, a1, a2, a3, qb[nt][g][2 * j], qb[nt][g][2 * j + 1]);
          }
          const float sa = pa.x * scale_log2, sb = pb.x * scale_log2;
          const float oa = fmaf(-128.f, sa, pa.y * scale_log2);
          const float ob = fmaf(-128.f, sb, pb.y * scale_log2);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            sc[k][nt][0] = fmaf(sa, acc[nt][0], fmaf(oa, qs[nt][g][0], sc[k][nt][0]));
            sc[k][nt][1] = fmaf(sa, acc[nt][1], fmaf(oa, qs[nt][g][1], sc[k][nt][1]));
            sc[k][nt][2] = fmaf(sb, acc[nt][2], fmaf(ob, qs[nt][g][0], sc[k][nt][2]));
            sc[k][nt][3] = fmaf(sb, acc[nt][3], fmaf(ob, qs[nt][g][1], sc[k][nt][3]));
          }
        }
      }
      // ---- mask: only where some row does not see the whole share
      if (k0 + 32 > kf.hi || k0 < kl.lo || (have & 3) != 3) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = k0 + k * kBlock + krow + (e / 2) * 8;
              if (!(have >> k & 1) || key < q_lo[nt][e % 2] || key >= q_hi[nt][e % 2])
                sc[k][nt][e] = -CUDART_INF_F;
            }
      }
      // ---- running maximum of each column over the warp's eight row groups
      float mx[NT][2];
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(fmaxf(sc[0][nt][e], sc[0][nt][e + 2]),
                          fmaxf(sc[1][nt][e], sc[1][nt][e + 2]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          mx[nt][e] = x;
          grow = grow || x > m[nt][e] + kTau;  // also the first finite maximum
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float corr[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mn = fmaxf(m[nt][e], mx[nt][e]);
            corr[e] = mn == -CUDART_INF_F ? 1.f : fast_exp2(m[nt][e] - mn);
            m[nt][e] = mn;
            l[nt][e] *= corr[e];
          }
#pragma unroll
          for (int i2 = 0; i2 < MT; ++i2) {
            o[nt][i2][0] *= corr[0];
            o[nt][i2][1] *= corr[1];
            o[nt][i2][2] *= corr[0];
            o[nt][i2][3] *= corr[1];
          }
        }
      }
      // ---- P = 2^(s - m) as fp16 B operands, and the values of each block
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float mm = m[nt][e % 2] == -CUDART_INF_F ? 0.f : m[nt][e % 2];
            p[e] = fast_exp2(sc[k][nt][e] - mm);
          }
          l[nt][0] += p[0] + p[2];
          l[nt][1] += p[1] + p[3];
          pb[nt][0] = transpose8(as_u32(__floats2half2_rn(p[0], p[1])));
          pb[nt][1] = transpose8(as_u32(__floats2half2_rn(p[2], p[3])));
        }
        if (!(have >> k & 1)) continue;
        const uint32_t vb = st + k * C::BLOCK_BYTES + value_offset(D);
        const uint32_t pairs = vb + code_bytes(D) + (r * NG / 8) * 4;  // the lane's group
        uint32_t pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pr[e] = lds32(pairs + (t + 4 * e) * NG * 4);
          // behind the last token the pairs may be anything: 0 times them must be 0
          if (k0 + k * kBlock + t + 4 * e >= s.w.L) pr[e] = 0u;
        }
        const __half2 step01 = as_half2(__byte_perm(pr[0], pr[1], 0x5410)),
                      lo01 = as_half2(__byte_perm(pr[0], pr[1], 0x7632)),
                      step23 = as_half2(__byte_perm(pr[2], pr[3], 0x5410)),
                      lo23 = as_half2(__byte_perm(pr[2], pr[3], 0x7632));
        uint32_t w[4][D / 64];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t at = vb + (t + 4 * e) * (D / 2) + r * (D / 16);
          if constexpr (D == 128) {
            const uint2 x = lds64(at);
            w[e][0] = x.x;
            w[e][1] = x.y;
          } else {
            w[e][0] = lds32(at);
          }
        }
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
#pragma unroll
          for (int hl = 0; hl < 2; ++hl) {  // four channels: D/8 lane / 4 + 8 j + 4 hl + 0..3
            uint32_t v01[4], v23[4];
            values4(__byte_perm(w[0][j], w[1][j], hl ? 0x7632 : 0x5410), step01, lo01, v01);
            values4(__byte_perm(w[2][j], w[3][j], hl ? 0x7632 : 0x5410), step23, lo23, v23);
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(o[nt][4 * j + 2 * hl + i2], v01[2 * i2], v01[2 * i2 + 1], v23[2 * i2],
                        v23[2 * i2 + 1], pb[nt][0], pb[nt][1]);
          }
      }
      __syncwarp();  // every lane has read the stage
      if (next < i1) issue(next++);
    }

    // ---- the four warps' partial softmaxes joined, in the accumulators' own layout
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nt][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (r == 0) {
          ml_s[(warp * TILE + 8 * nt + 2 * t + e) * 2] = m[nt][e];
          ml_s[(warp * TILE + 8 * nt + 2 * t + e) * 2 + 1] = x;
        }
      }
    // merge[warp][tile nt and M tile i][lane] as float4
    float4* mg = reinterpret_cast<float4*>(merge);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i2 = 0; i2 < MT; ++i2)
        mg[(warp * NT * MT + nt * MT + i2) * 32 + lane] =
            make_float4(o[nt][i2][0], o[nt][i2][1], o[nt][i2][2], o[nt][i2][3]);
    __syncthreads();
    const bool whole = s.first && s.last;
    const long long slot = 2ll * blockIdx.x + (s.first ? 1 : 0);
    // warp w joins the M tiles w MT / 4 ..: lane (r, t) holds channels D/8 r + 2 i, + 1 of
    // query rows 2 t, 2 t + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[kWarps][2], mt[2], lt[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int n = 8 * nt + 2 * t + e;
        mt[e] = -CUDART_INF_F;
        lt[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mt[e] = fmaxf(mt[e], ml_s[(w * TILE + n) * 2]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          f[w][e] = mt[e] == -CUDART_INF_F ? 0.f : fast_exp2(ml_s[(w * TILE + n) * 2] - mt[e]);
          lt[e] = fmaf(f[w][e], ml_s[(w * TILE + n) * 2 + 1], lt[e]);
        }
      }
      float x[2][MT / 2];  // [row][channel] of the warp's MT / 4 tiles
#pragma unroll
      for (int i2 = 0; i2 < MT / 4; ++i2) {
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 v = mg[(w * NT * MT + nt * MT + warp * (MT / 4) + i2) * 32 + lane];
          sum.x = fmaf(f[w][0], v.x, sum.x);
          sum.y = fmaf(f[w][1], v.y, sum.y);
          sum.z = fmaf(f[w][0], v.z, sum.z);
          sum.w = fmaf(f[w][1], v.w, sum.w);
        }
        x[0][2 * i2] = sum.x;
        x[0][2 * i2 + 1] = sum.z;
        x[1][2 * i2] = sum.y;
        x[1][2 * i2 + 1] = sum.w;
      }
      const int ch = r * (D / 8) + warp * (MT / 2);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int n = 8 * nt + 2 * t + e;
        if (n >= rows) continue;
        if (whole) {
          const long long row = row0 + n;
          const long long at = (s.w.q0 + row / G) * c.Hq + (long long)s.h * G + row % G;
          const float inv = lt[e] > 0.f ? 1.f / lt[e] : 0.f;
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + at * D + ch;
#pragma unroll
          for (int k = 0; k < MT / 4; ++k)
            reinterpret_cast<uint32_t*>(dst)[k] =
                pack_bf16x2(x[e][2 * k] * inv, x[e][2 * k + 1] * inv);
          if (warp == 0 && r == 0) a.lse[at] = (mt[e] + log2f(lt[e])) * 0.6931471805599453f;
        } else {
          const long long at = slot * a.tile + n;
          float* dst = a.acc + at * D + ch;
#pragma unroll
          for (int k = 0; k < MT / 4; ++k)
            reinterpret_cast<float2*>(dst)[k] = make_float2(x[e][2 * k], x[e][2 * k + 1]);
          if (warp == 0 && r == 0) {
            a.ml[at * 2] = mt[e];
            a.ml[at * 2 + 1] = lt[e];
          }
        }
      }
    }
    if (s.followers) followers = s.followers, fb = s.b, fh = s.h, ft = s.tile;
    __syncthreads();
  }
  if (threadIdx.x == 0) a.desc[blockIdx.x] = PartDesc{followers, fb, fh, ft};
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // copies of a share that was never consumed (after an expired wait) must land before the
  // block's shared memory goes away
  int dummy = 0;
  for (; consumed != issued; ++consumed)
    if (!mbar_wait_warp(&bar[consumed % kStages], (consumed / kStages) & 1, &dummy, a.err,
                        K_CACHE_ATTN, 2, a.wait_ns))
      break;
}

template <int D, int NT>
cudaError_t launch(const AttnArgs& a, int* blocks, cudaStream_t s) {
  using C = RowsCfg<D, NT>;
  const cudaError_t e = cudaFuncSetAttribute(
      cache_attn_rows_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  *blocks = kSms * C::CTAS;  // one wave
  cache_attn_rows_kernel<D, NT><<<*blocks, kThreads, C::SMEM, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_rows(AttnArgs& a, long long rows, int* blocks, cudaStream_t s) {
  a.tile = rows <= 8 ? 8 : 16;
  if (rows <= 8) return a.c.d == 64 ? launch<64, 1>(a, blocks, s) : launch<128, 1>(a, blocks, s);
  return a.c.d == 64 ? launch<64, 2>(a, blocks, s) : launch<128, 2>(a, blocks, s);
}

}  // namespace ra
