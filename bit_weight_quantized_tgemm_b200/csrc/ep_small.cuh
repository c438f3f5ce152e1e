// ep_small.cuh -- the epilogue and expert matmuls for a few rows per expert (warp MMA).
//
// Item: an expert's chunk of up to 8 T rows x 32 weight rows, the whole of K.  A CTA takes a
// run of neighbouring items; its 8 warps split K in units of 128 weights, each a contiguous
// share, and their f32 sums meet in shared memory, are added in warp order and go through the
// epilogue.  One barrier an item: the sums have two buffers.
//
// Weights come straight from global memory into registers, kD units ahead and across items:
// lane (g, c) of mma.sync m16n8k16 takes weight rows g + 8 j and, in each 32-byte sector of a
// row, bytes [8c, 8c + 8).  The codes in there and the activations they meet are the same k for
// every row, so nothing moves between lanes.  (The buffers are named, not shifted: moving a
// register waits for the load that fills it.)
// Activations stay the same over a run of items of one expert: each lane keeps its own B
// fragments in shared memory, already paired as the codes unpack.
// Scales come by asynchronous copies of 32-bit words, an item ahead, 8 rows x 4 words at a
// time; read row by row each unit they would touch 32 lines.
//
// A word of codes becomes bf16 pairs of whole numbers: one lop3 sets an exponent over a field
// (base + q), one subtraction takes off the base and the centre, q - 1 (ternary) or q - 8
// (4-bit).  Products with bf16 activations are exact; per 128 (64) weights the f32 sum is
// scaled, and 4-bit adds the zero point by the sum of the activations (an MMA with ones):
//   ternary  acc += d * sum (q - 1) x
//   4-bit    acc += s * (sum (q - 8) x - (z - 8) sum x)
//
// What bounds it: latency.  One token x 2560 x 2560 ternary, 1.8 MB, takes 4.1 us in a chain of calls
// (0.4 TB/s), of which 3 us are there at any size; 8 tokens x 9728 x 2560 ternary 7.9 us
// (0.8 TB/s), 4-bit 10.7 us (1.3 TB/s, twice the bytes).  Counters of these two, cold: 39 and 37 % of
// the issue slots used, ALU 28 %, tensor pipe 10 and 12 %, and the warps wait for global loads more
// than for anything else (3.2 and 2.7 warps for each instruction issued).
// A warp's units follow each other at 0.6 to 1.4 us, so that long rows with few items go to
// clusters (SHARE): one token x 1408 x 9728 4-bit 14.1 -> 6.5 us.
#pragma once

#include "common.cuh"
#include "ep_tc.cuh"
#include "epilogue.cuh"
#include "gemv_stream.cuh"

namespace tgemm {

constexpr int kEsWarps = 8;
constexpr int kEsRows = 32;   // weight rows of an item
constexpr int kEsPitch = 36;  // floats per token row of a warp's sums: no bank conflicts

struct EsParams {
  int N, K, E, R, x_rows;
  int U;        // units of 128 k
  int tiles_n;  // blocks of 32 weight rows
  int nu_max;   // most units of a warp
  int split;    // CTAs of a cluster that share an item's K (dense calls)
  int staged;   // activations kept in shared memory (else read from global each unit)
  const uint16_t* x;
  const uint8_t* wq;
  const uint16_t* scales;
  const int* offsets;
  const int* rows;
  EpArgs ep;
};

// Scale words of a row that a warp's units can take: Q2 two blocks a word, 4-bit two words a unit.
__host__ __device__ constexpr int es_words(int fmt, int nu) { return (fmt == 0 ? nu / 2 + 1 : 2 * nu) + 3 & ~3; }
// two buffers of the warps' sums, or one and the sums of a cluster's CTAs
__host__ __device__ constexpr int es_red_bytes(int T, bool share) {
  return (kEsWarps * kEsPitch + (share ? kEtMaxSplit * kEsRows : kEsWarps * kEsPitch)) * 8 * T * 4;
}
__host__ __device__ constexpr int es_scale_bytes(int fmt, int nu) { return kEsWarps * 2 * es_words(fmt, nu) * 128; }
__host__ __device__ constexpr int es_x_bytes(int T, int nu) { return kEsWarps * nu * T * 2048; }
__host__ __device__ constexpr int es_smem_bytes(int fmt, int T, bool share, int nu, bool staged, int E, bool grouped) {
  return es_red_bytes(T, share) + es_scale_bytes(fmt, nu) + (staged ? es_x_bytes(T, nu) : 0) + (grouped ? 2 * (E + 2) * 4 : 0);
}

__device__ __forceinline__ uint2 ld_stream_v2(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t bsub2_u32(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// A lane's codes of one unit: rows g + 8 j.
template <int FMT>
struct EsUnit {
  static constexpr int kW = FMT == 0 ? 2 : 4;  // 32-bit words of codes per row
  uint32_t w[4][kW];
};

// SHARE: the warps of a cluster's CTAs share the K of one item; CTA 0 adds the CTAs' sums in order.
template <int FMT, int T, bool SHARE>
__global__ void __launch_bounds__(kEsWarps * 32, 2) ep_small_kernel(const EsParams p) {
  constexpr int kTok = 8 * T;
  constexpr int kUnitBytes = FMT == 0 ? 32 : 64;
  constexpr int kD = FMT == 0 ? 3 : 2;  // units in flight
  using Unit = EsUnit<FMT>;
  extern __shared__ __align__(16) uint8_t es_smem[];
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x) >> 5, 0);
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  float* red = reinterpret_cast<float*>(es_smem);  // [buffer][warp][token][kEsPitch]
  const int words = es_words(FMT, p.nu_max);
  uint8_t* sc_base = es_smem + es_red_bytes(T, SHARE);
  uint4* sc_mine = reinterpret_cast<uint4*>(sc_base) + warp * 2 * words * 8;   // [buffer][word][8 g][4 j]
  uint4* xs_mine = reinterpret_cast<uint4*>(sc_base + es_scale_bytes(FMT, p.nu_max)) +
                   warp * p.nu_max * T * 128 + lane;                            // [unit][tile][4][lane]
  int* tab_off = reinterpret_cast<int*>(sc_base + es_scale_bytes(FMT, p.nu_max) +
                                        (p.staged ? es_x_bytes(T, p.nu_max) : 0));
  int* tab_tp = tab_off + p.E + 2;
  const int row_bytes = FMT == 0 ? p.K / 4 : p.K / 2;
  const int nscale = FMT == 0 ? p.K / 128 : p.K / 64;
  const int split = SHARE ? p.split : 1, rank = static_cast<int>(blockIdx.x) % split;
  const int cta = static_cast<int>(blockIdx.x) / split, ctas = static_cast<int>(gridDim.x) / split;
  const int part = rank * kEsWarps + warp, parts = split * kEsWarps;
  const int ua = p.U * part / parts, ub = p.U * (part + 1) / parts, nu = ub - ua;

  pdl_trigger();
  if (SHARE) cluster_arrive();  // CTA 0 is there to be written to
  int num_items;
  const int chunks = (p.R + kTok - 1) / kTok;  // dense
  if (p.offsets) {
    pdl_wait();
    if (warp == 0) et_build_table(p.offsets, p.E, p.R, kTok, tab_off, tab_tp);
    __syncthreads();
    num_items = tab_tp[p.E] * p.tiles_n;
  } else {
    num_items = chunks * p.tiles_n;
  }
  // this CTA's items
  const int t0 = static_cast<int>(static_cast<int64_t>(num_items) * cta / ctas);
  const int t1 = static_cast<int>(static_cast<int64_t>(num_items) * (cta + 1) / ctas);
  struct Item {
    int e, n0, m0, mt;
  };
  auto item_at = [&](int t) {  // chunk by chunk, row block by row block
    Item it;
    it.e = 0;
    int ch = t / p.tiles_n, lo = 0, hi = p.R;
    it.n0 = (t - ch * p.tiles_n) * kEsRows;
    if (p.offsets) {
      it.e = et_find(tab_tp, p.E, ch);
      ch -= tab_tp[it.e];
      lo = tab_off[it.e];
      hi = tab_off[it.e + 1];
    }
    it.m0 = lo + ch * kTok;
    it.mt = min(kTok, hi - it.m0);
    return it;
  };
  auto w_at = [&](const Item& it) {
    return p.wq + (static_cast<int64_t>(it.e) * p.N + it.n0) * row_bytes + static_cast<int64_t>(ua) * kUnitBytes + 8 * c;
  };
  // unit j of the warp's share of the item whose codes start at `base`; rows past N read row
  // N - 1 (their sums are not stored)
  auto load_unit = [&](Unit& b, const uint8_t* base, int last, int j) {
    const uint8_t* src = base + j * kUnitBytes;
    const bool second = FMT == 1 && 2 * (ua + j) + 1 < nscale;  // K may end on half a unit
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint8_t* q = src + static_cast<int64_t>(min(g + 8 * r, last)) * row_bytes;
      const uint2 v = ld_stream_v2(q);
      b.w[r][0] = v.x;
      b.w[r][1] = v.y;
      if (FMT == 1) {
        const uint2 h = second ? ld_stream_v2(q + 32) : make_uint2(0u, 0u);
        b.w[r][Unit::kW - 2] = h.x;
        b.w[r][Unit::kW - 1] = h.y;
      }
    }
  };
  // The warp's scales of an item -> buffer `buf`: word w of row g + 8 j at [w][g][j].
  // Q2 scales are words of two blocks; where rows do not start on words, by plain loads.
  const int wbase = FMT == 0 ? ua >> 1 : 2 * ua;
  const int nwords = FMT == 0 ? (nu ? ((ub - 1) >> 1) - wbase + 1 : 0) : min(2 * ub, nscale) - wbase;
  const bool even = FMT == 1 || ((nscale & 1) == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 3) == 0);
  auto load_scales = [&](const Item& it, int buf) {
    const int last = p.N - 1 - it.n0;
    const int64_t row0 = static_cast<int64_t>(it.e) * p.N + it.n0;
    uint4* dst = sc_mine + buf * words * 8;
    for (int w = lane & 3; w < nwords; w += 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t row = row0 + min((lane >> 2) + 8 * j, last);
        uint32_t* d = reinterpret_cast<uint32_t*>(dst + w * 8 + (lane >> 2)) + j;
        if (even) {
          const uint32_t* src = reinterpret_cast<const uint32_t*>(p.scales) +
                                (FMT == 0 ? row * (nscale / 2) : row * nscale) + wbase + w;
          cp_async4(smem_u32(d), src, 4u);
        } else {
          const uint16_t* src = p.scales + row * nscale + 2 * (wbase + w);
          uint32_t v = ld_scale(src);
          if (2 * (wbase + w) + 1 < nscale) v |= static_cast<uint32_t>(ld_scale(src + 1)) << 16;
          *d = v;
        }
      }
    }
  };
  // B fragments of one (unit, token tile, half): 16 activations of token g + 8 i as pairs
  auto x_frag = [&](const uint16_t* src, bool ok, uint32_t (&b)[8]) {
    const uint4* xs = reinterpret_cast<const uint4*>(src);
    uint4 r0 = make_uint4(0u, 0u, 0u, 0u), r1 = r0;
    if (ok) {
      r0 = xs[0];
      r1 = xs[1];
    }
    const uint32_t r[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {  // codes (i, i + 8), or (i, i + 4) of each word
      const int lo = FMT == 0 ? k / 2 : 4 * (k / 4) + (k & 3) / 2;
      b[k] = prmt(r[lo], r[lo + (FMT == 0 ? 4 : 2)], (k & 1) ? 0x7632u : 0x5410u);
    }
  };

  Unit buf[kD];
  Item cur{0, 0, 0, 0};
  const uint8_t* wcur = nullptr;
  if (t0 < t1) {
    cur = item_at(t0);
    wcur = w_at(cur);
#pragma unroll
    for (int d = 0; d < kD; ++d)
      if (d < nu) load_unit(buf[d], wcur, p.N - 1 - cur.n0, d);
    load_scales(cur, 0);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  if (!p.offsets) pdl_wait();

  const uint16_t* xp[T];
  bool xok[T];
  int have_m0 = -1;
  for (int t = t0; t < t1; ++t) {
    Item nxt = cur;
    const uint8_t* wnxt = wcur;
    const bool more = t + 1 < t1;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    const uint4* sc_cur = sc_mine + ((t - t0) & 1) * words * 8 + g;
    if (more) {
      nxt = item_at(t + 1);
      wnxt = w_at(nxt);
      load_scales(nxt, (t - t0 + 1) & 1);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (cur.m0 != have_m0) {
      // the lane's token rows: row g + 8 i of the chunk (past its end: its last), the elements
      // that meet the lane's 8 (Q2) or 2 x 8 (4-bit) bytes of a unit
      have_m0 = cur.m0;
#pragma unroll
      for (int i = 0; i < T; ++i) {
        int64_t m = cur.m0 + min(g + 8 * i, cur.mt - 1);
        if (p.rows) m = p.rows[m];
        xok[i] = m >= 0 && m < p.x_rows;  // else a row of zeros
        xp[i] = p.x + (xok[i] ? m : 0) * p.K + static_cast<int64_t>(ua) * 128 + (FMT == 0 ? 32 : 16) * c;
      }
      if (p.staged) {
        for (int j = 0; j < nu; ++j)
#pragma unroll
          for (int i = 0; i < T; ++i)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              uint32_t b[8];
              x_frag(xp[i] + j * 128 + (FMT == 0 ? 16 : 64) * hf,
                     xok[i] && (FMT == 0 || 2 * (ua + j) + hf < nscale), b);
              uint4* dst = xs_mine + ((j * T + i) * 4 + 2 * hf) * 32;
              dst[0] = make_uint4(b[0], b[1], b[2], b[3]);
              dst[32] = make_uint4(b[4], b[5], b[6], b[7]);
            }
      }
    }
    float acc[2][T][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[h][i][k] = 0.f;

    for (int j0 = 0; j0 < nu; j0 += kD) {
#pragma unroll
      for (int d = 0; d < kD; ++d) {
        const int j = j0 + d;
        if (j >= nu) break;
        const Unit& cu = buf[d];
        float pacc[2][T][4];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {  // Q2: two half units under one scale; 4-bit: two groups
          if (FMT == 1 && 2 * (ua + j) + hf >= nscale) break;
          if (FMT == 1 || hf == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < T; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) pacc[h][i][k] = 0.f;
          }
          float xsum[T][4];
          uint32_t a[4][8];  // bf16 pairs of 16 codes per row
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (FMT == 0) {
              gs_q2_pairs(cu.w[r][hf], a[r]);
              constexpr uint32_t kOne[3] = {0x43014301u, 0x42044204u, 0x41104110u};  // 129, 33, 9
#pragma unroll
              for (int i = 0; i < 8; ++i) a[r][i] = bsub2_u32(a[r][i], kOne[i % 3]);
            } else {
#pragma unroll
              for (int wd = 0; wd < 2; ++wd)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  a[r][4 * wd + i] =
                      bsub2_u32(lop3_and_or(cu.w[r][(2 * hf + wd) % Unit::kW] >> (4 * i), 0x000F000Fu, 0x43004300u),
                                0x43084308u);  // 136
            }
          }
#pragma unroll
          for (int i = 0; i < T; ++i) {
            uint32_t b[8];
            if (p.staged) {
              const uint4* src = xs_mine + ((j * T + i) * 4 + 2 * hf) * 32;
              const uint4 b0 = src[0], b1 = src[32];
              b[0] = b0.x; b[1] = b0.y; b[2] = b0.z; b[3] = b0.w;
              b[4] = b1.x; b[5] = b1.y; b[6] = b1.z; b[7] = b1.w;
            } else {
              x_frag(xp[i] + j * 128 + (FMT == 0 ? 16 : 64) * hf, xok[i], b);
            }
            if (FMT == 1) {
#pragma unroll
              for (int k = 0; k < 4; ++k) xsum[i][k] = 0.f;
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t af[4] = {a[2 * h][2 * s], a[2 * h + 1][2 * s], a[2 * h][2 * s + 1], a[2 * h + 1][2 * s + 1]};
                mma_bf16_16816(pacc[h][i], af, b[2 * s], b[2 * s + 1]);
              }
              if (FMT == 1) {
                const uint32_t ones[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
                mma_bf16_16816(xsum[i], ones, b[2 * s], b[2 * s + 1]);
              }
            }
          }
          if (FMT == 0 && hf == 0) continue;
          const uint4 sw = sc_cur[(FMT == 0 ? ((ua + j) >> 1) - wbase : 2 * j + hf) * 8];
          const uint32_t sv[4] = {sw.x, sw.y, sw.z, sw.w};
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint32_t v = FMT == 0 && ((ua + j) & 1) ? sv[r] >> 16 : sv[r];
            const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(v & 0xFFFFu)));
            const int h = r >> 1, k0 = 2 * (r & 1);
            if (FMT == 0) {
#pragma unroll
              for (int i = 0; i < T; ++i) {
                acc[h][i][k0] = fmaf(s, pacc[h][i][k0], acc[h][i][k0]);
                acc[h][i][k0 + 1] = fmaf(s, pacc[h][i][k0 + 1], acc[h][i][k0 + 1]);
              }
            } else {
              const float z = __half2float(__ushort_as_half(static_cast<uint16_t>(v >> 16))) - 8.f;
#pragma unroll
              for (int i = 0; i < T; ++i) {
                acc[h][i][k0] = fmaf(s, fmaf(-z, xsum[i][0], pacc[h][i][k0]), acc[h][i][k0]);
                acc[h][i][k0 + 1] = fmaf(s, fmaf(-z, xsum[i][1], pacc[h][i][k0 + 1]), acc[h][i][k0 + 1]);
              }
            }
          }
        }
        // the buffer's next unit: of this item, or its first of the next item
        if (j + kD < nu)
          load_unit(buf[d], wcur, p.N - 1 - cur.n0, j + kD);
        else if (more)
          load_unit(buf[d], wnxt, p.N - 1 - nxt.n0, d);
      }
    }
    // ---- sums of the warps -> epilogue.  acc[h][i][k]: weight row 16 h + g (+ 8 for k >= 2),
    // token 8 i + 2 c + (k & 1)
    float* rb = red + ((t - t0) & 1) * kEsWarps * kTok * kEsPitch;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          rb[(warp * kTok + 8 * i + 2 * c + (k & 1)) * kEsPitch + 16 * h + g + 8 * (k >> 1)] = acc[h][i][k];
    __syncthreads();
    const int n = cur.n0 + lane;
    if constexpr (SHARE) {
      // the cluster's only item (the grid has one cluster for each); CTA 0 gets the sums
      // [CTA][token][32 rows]
      float* all = red + kEsWarps * kTok * kEsPitch;
      cluster_wait();
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const int m = warp + kEsWarps * i;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kEsWarps; ++w) v += rb[(w * kTok + m) * kEsPitch + lane];
        st_cluster_f32(smem_u32(all + (rank * kTok + m) * kEsRows + lane), 0, v);
      }
      cluster_sync();
      if (rank > 0) break;
      if (n < p.N) {
        float bias = 0.f;
        if (p.ep.bias) bias = ep_load(p.ep.bias, n, p.ep.bias_f32);
        for (int m = warp; m < cur.mt; m += kEsWarps) {
          float v[1] = {0.f};
          for (int r = 0; r < split; ++r) v[0] += all[(r * kTok + m) * kEsRows + lane];
          v[0] += bias;
          ep_act_all(v, p.ep.act);
          ep_store1(p.ep, cur.m0 + m, n, p.N, v[0]);
        }
      }
    } else if (n < p.N) {
      float bias = 0.f;
      if (p.ep.bias) bias = ep_load(p.ep.bias, static_cast<int64_t>(cur.e) * p.N + n, p.ep.bias_f32);
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const int m = warp + kEsWarps * i;
        if (m >= cur.mt) break;
        float v[1] = {0.f};
#pragma unroll
        for (int w = 0; w < kEsWarps; ++w) v[0] += rb[(w * kTok + m) * kEsPitch + lane];
        v[0] += bias;
        ep_act_all(v, p.ep.act);
        ep_store1(p.ep, cur.m0 + m, n, p.N, v[0]);
      }
    }
    cur = nxt;
    wcur = wnxt;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace tgemm
