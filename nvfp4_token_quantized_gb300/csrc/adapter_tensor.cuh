// adapter_tensor.cuh - rows through their adapters (as adapter_apply.cuh) for
// batches of many rows: both products on the tensor cores' tcgen05 path, operands
// in 128-byte swizzled shared memory, sums in tensor memory.
//
// A tile is 128 rows of one adapter.  Its x is streamed in stages of 64 columns
// beside the same columns of down (D1 += x down^T, 128 x rank), then base and up in
// stages of 64 output columns (D2 = hidden up, 128 x 64).  The rows are those that
// the plan lists, in any order, so they come by 16-byte asynchronous copies, each
// to the place that the swizzle gives it; up is read as it lies, rank rows of
// neighbouring columns, which is the layout of an operand whose columns are
// contiguous.  hidden enters the second product as two 16-bit parts side by side
// (split2), which doubles a contraction of 16 to 128 and costs nothing visible.
//
// Rows that do not start on 16 bytes (or widths that are no multiple of 8) are read
// as aligned words one stage ahead, put in order in registers and stored to the
// same places; their output leaves element by element.
//
// Eight warps copy (and later add and store); a ninth issues a stage's products when
// all copies of the stage have arrived on its barrier, and their commit frees the
// slot.  Two CTAs share an SM, so that the join between one's products hides behind
// the other's copies.  The CTAs of a cluster split a tile as in adapter_apply.cuh.
// Rows behind a tile's last are not copied: what lies in their places gives rows
// that are not stored.
//
// Bound by bytes: x once, base and out once, and from L2 the factors once a tile
// (as many as x and base again at rank 128).  16384 rows, 4096 to 4096, eight
// adapters, bf16: rank 16 79 us, 32 81, 64 89, 128 126 for 403 MB (60 us at a copy's
// rate); of the 89 the plan takes 4, the first product 28, the join 8, the second
// product 43.  The join is distributed shared memory's: every CTA sums a share of
// the rows and sends it to the others (gathering all of them everywhere took up to
// twice the kernel's time at eight CTAs, and lanes of a warp that read several CTAs
// at once a tenth more).  65536 rows, rank 64: 305 us (241).  Rows of odd alignment
// take twice the time (16384 rows, 4095 to 4097, rank 16: 180 us).
//
// Two of these CTAs at most share an SM, or one beside a CTA of the gradients'
// kernel (registers, shared memory), and the layer's GEMMs leave no room beside
// theirs: tensor memory is never waited for.
//
// Waits are bounded: after one that runs out the CTA issues and copies no more, what is
// on its way ends before shared memory changes its use and before tensor memory is
// given back, and the tile's rows become NaN: all of them in every CTA of the cluster
// where the first product is incomplete, else the CTA's columns from there on.
#pragma once

#include <cooperative_groups.h>

#include "adapter_common.cuh"
#include "adapter_mma.cuh"

namespace moe {
namespace cg = cooperative_groups;

template <int R>
struct TensorShared {
  static constexpr int ROWS = ADAPTER_TILE * 128;          // of x, or of base and out
  static constexpr int STAGE = ROWS + R * 128;
  static constexpr int STAGES = R == 64 ? 3 : 4;
  static constexpr int PANELS = R <= 32 ? 1 : 2 * R / 64;  // of hidden's parts, 64 wide
  static constexpr int RP = hidden_pitch(R);
  static constexpr int HIDDEN = PANELS * ROWS;
  static constexpr int BYTES = HIDDEN + STAGES * STAGE + 1024;  // (aligned inside)
  static_assert(ADAPTER_TILE * RP * 4 <= STAGES * STAGE, "the first product's sums lie in the stages");
};

template <typename T, int R, bool VEC>
__global__ void __launch_bounds__(TENSOR_THREADS, R <= 64 ? 2 : 1) adapter_tensor_kernel(const AdapterArgs a) {
  using S = TensorShared<R>;
  constexpr int ST = S::STAGES, RP = S::RP, W = (R + 31) / 32;  // (a thread's chunks of a factor)
  constexpr int SUMS = 4;  // stages whose sums tensor memory holds
  constexpr bool SCALED = !std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ unsigned char raw[];
  unsigned char* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  unsigned char* panels = smem;                 // hidden's parts
  unsigned char* ring = smem + S::HIDDEN;
  float* part = reinterpret_cast<float*>(ring);  // (between the products)
  __shared__ int row_of[ADAPTER_TILE];
  __shared__ int64_t base_at[ADAPTER_TILE], out_at[ADAPTER_TILE];  // the rows' first elements
  __shared__ float back[ADAPTER_TILE];
  __shared__ Piece found;
  // Of the first product's slots: copies in, products done; of the second's: copies
  // in; of D2's SUMS places: products done, sums read.
  __shared__ uint64_t in1[ST], free1[ST], in2[ST], done[SUMS], drained[SUMS];
  __shared__ uint64_t last;  // (nothing arrives but after a wait that ran out)
  __shared__ uint32_t tmem_at;
  __shared__ volatile int gave_up;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool issuer = warp == ADAPTER_WARPS;
  const int C = a.cluster, crank = blockIdx.x % C, number = blockIdx.x / C;

  // Of many adapters most numbers are unused, and leave before they take anything.
  Piece p;
  if (a.group_of) {
    pdl_wait();
    p = find_piece(a.starts, a.rows, a.groups, ADAPTER_TILE, number, &found);
    if (p.group < 0) return;  // (the whole cluster)
  }
  // (set up while the plan is made)
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&in1[i], ADAPTER_THREADS);
      mbar_init(&in2[i], ADAPTER_THREADS / 2);
      mbar_init(&free1[i], 1);
    }
    for (int i = 0; i < SUMS; ++i) {
      mbar_init(&done[i], 1);
      mbar_init(&drained[i], ADAPTER_WARPS / 2);
    }
    mbar_init(&last, 1);
    gave_up = 0;
    fence_mbarrier_init();
  }
  if (warp == 0) {
    tmem_alloc(&tmem_at, SUMS * 64);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at, ring_at = smem_u32(ring), panels_at = smem_u32(panels);
  if (!a.group_of) {
    pdl_wait();
    p = find_piece(a.starts, a.rows, a.groups, ADAPTER_TILE, number, &found);
  }
  pdl_trigger();
  if (p.group < 0) {  // (the whole cluster)
    if (warp == 0) tmem_dealloc(tmem, SUMS * 64);
    return;
  }
  const int count = p.count, group = a.group_of ? a.group_of[p.group] : p.group;  // (the adapter)
  if (tid < ADAPTER_TILE) {
    const int row = tid < count ? a.row_list[p.start + tid] : 0;
    row_of[tid] = row;
    base_at[tid] = row * a.base_stride;
    out_at[tid] = row * a.out_stride;
    back[tid] = 1.0f;
  }
  const T* x = static_cast<const T*>(a.x);
  const T* base = static_cast<const T*>(a.base);
  T* out = static_cast<T*>(a.out);
  const int K = a.in, N = a.n_out;
  __syncthreads();
  if (group == a.L) {
    if (warp == 0) tmem_dealloc(tmem, SUMS * 64);
    if (!issuer) rows_without_adapter<T, VEC>(a, row_of, count, crank, C);
    return;
  }
  const Waits wait(&gave_up, a.silent);

  // ---- D1 = x down^T over this CTA's columns ----
  const int chunks = (K + 63) / 64, each = (chunks + C - 1) / C;
  const int c0 = min(crank * each, chunks), nk = min(each, chunks - c0);
  const int blocks = (N + 63) / 64, blocks_each = (blocks + C - 1) / C;  // (of the second product)
  const int b0 = min(crank * blocks_each, blocks), nb = min(blocks_each, blocks - b0);
  if (issuer) {
    if (lane == 0)
      for (int i = 0; i < nk; ++i) {
        if (!wait.alone(i == 0 && crank + 1 == a.silent ? &last : &in1[i % ST], (i / ST) & 1)) break;
        fence_async_shared();
        const uint32_t at = ring_at + (i % ST) * S::STAGE;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_f16(tmem, smem_desc_sw128(at + k * 32), smem_desc_sw128(at + S::ROWS + k * 32),
                     idesc_f16<T>(R, false, false), i > 0 || k > 0);
        tc_commit(&free1[i % ST]);
      }
    __syncwarp();
  } else {
    const int sub = tid & 7, r0 = tid >> 3;  // 16-byte chunk of a row, first of the rows 32 apart
    const T* px[4];
    bool on[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      on[i] = r0 + 32 * i < count;
      px[i] = x + (int64_t)row_of[r0 + 32 * i] * a.x_stride;
    }
    const T* down = static_cast<const T*>(a.first) + (int64_t)group * a.rank * K;
    const auto issue = [&](int i) {
      const uint32_t at = ring_at + (i % ST) * S::STAGE;
      const bool in = (c0 + i) * 64 + sub * 8 < K;
      const int col = in ? (c0 + i) * 64 + sub * 8 : 0;  // (a copy of nothing has an address all the same)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (on[q]) copy16(at + swizzled(r0 + 32 * q, sub), px[q] + col, in);
#pragma unroll
      for (int r = r0; r < R; r += 32) {
        const bool have = r < a.rank;
        copy16(at + S::ROWS + swizzled(r, sub), down + (have ? r * K : 0) + col, in && have);
      }
    };
    Loose lx[VEC ? 1 : 4], lw[VEC ? 1 : W];
    const auto fetch = [&](int i) {  // (rows that start anywhere)
      const int col = (c0 + i) * 64 + sub * 8;
#pragma unroll
      for (int q = 0; q < 4; ++q) lx[q].load(px[q] + col, K - col, on[q]);
#pragma unroll
      for (int q = 0; q < W; ++q) {
        const int r = r0 + 32 * q;
        lw[q].load(down + (int64_t)r * K + col, K - col, r < a.rank);
      }
    };
    const auto put = [&](int i) {
      const int col = (c0 + i) * 64 + sub * 8;
      const uint32_t at = ring_at + (i % ST) * S::STAGE;
#pragma unroll
      for (int q = 0; q < 4; ++q) put16(at + swizzled(r0 + 32 * q, sub), lx[q].chunk(Loose::odd(px[q] + col), K - col));
#pragma unroll
      for (int q = 0; q < W; ++q) {
        const int r = r0 + 32 * q;
        if (r < R) put16(at + S::ROWS + swizzled(r, sub), lw[q].chunk(Loose::odd(down + (int64_t)r * K + col), K - col));
      }
    };
    if (!VEC && nk > 0) fetch(0);
    for (int i = 0; i < nk; ++i) {
      if (i >= ST && !wait.warp(&free1[i % ST], ((i - ST) / ST) & 1)) break;
      if constexpr (VEC) {
        issue(i);
        copy_arrive(&in1[i % ST]);
      } else {
        put(i);
        if (i + 1 < nk) fetch(i + 1);
        mbar_arrive(&in1[i % ST]);
      }
    }
    if (nk > 0) wait.warp(&free1[(nk - 1) % ST], ((nk - 1) / ST) & 1);  // (the last commit covers all before)
  }
  __syncthreads();
  const bool lost = gave_up;  // (the same in all threads: none waits before the next barrier)
  if (lost) wait.settle(&last, 0, issuer && lane == 0);
  tc_fence_after();

  const int quarter = warp & 3, half = (warp >> 2) & 1, mine = quarter * 32 + lane;  // (the issuer takes no part)

  // ---- the cluster's sums joined, hidden's parts into every CTA's panels ----
  // (sums that this CTA could not form are no numbers: the join carries them into
  // hidden, every CTA's columns and the factors' gradients)
  if (!issuer) {
    float* to = part + mine * RP + half * (R / 2);
#pragma unroll
    for (int c = 0; c < R / 2; c += 8) {
      float v[8];
      if (nk > 0 && !lost) {
        tmem_ld8(tmem + ((uint32_t)(quarter * 32) << 16) + half * (R / 2) + c, v);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = lost ? NAN : 0.0f;
      }
      reinterpret_cast<float4*>(to + c)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(to + c)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    tc_fence_before();
  }
  cg::cluster_group cluster = cg::this_cluster();
  if (C > 1)
    cluster.sync();
  else
    __syncthreads();
  if (!issuer) {
    constexpr int G = R / 8;  // lanes of a row, eight ranks each
    const float scale = a.scales ? a.scales[group] : 1.0f;
    const int share = ADAPTER_TILE / C, lane8 = tid % G;
    for (int r = crank * share + tid / G; r < (crank + 1) * share; r += ADAPTER_THREADS / G) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
      for (int q0 = 0; q0 < C; q0 += 4) {  // (four CTAs' sums on their way together)
        float4 f[4][2];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int from = (crank + (q0 + q < C ? q0 + q : q0)) % C;  // (each begins at its own)
          const float4* p =
              reinterpret_cast<const float4*>((from != crank ? cluster.map_shared_rank(part, from) : part) + r * RP + lane8 * 8);
          f[q][0] = p[0], f[q][1] = p[1];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q0 + q < C) {
            v[0] += f[q][0].x, v[1] += f[q][0].y, v[2] += f[q][0].z, v[3] += f[q][0].w;
            v[4] += f[q][1].x, v[5] += f[q][1].y, v[6] += f[q][1].z, v[7] += f[q][1].w;
          }
      }
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // (nothing for the ranks that fill up: an infinite x times their zeros is none)
        v[i] = lane8 * 8 + i < a.rank ? v[i] * scale : 0.0f;
        m = fmaxf(m, fabsf(v[i]));
      }
      if (a.hidden && r < count) {
        float* h = a.hidden + (int64_t)row_of[r] * a.rank + lane8 * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (lane8 * 8 + i < a.rank) h[i] = v[i];
      }
      float s = 1.0f, b = 1.0f;
      if constexpr (SCALED) {
#pragma unroll
        for (int o = 1; o < G; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        s = exponent_scale(m, b);
      }
      uint4 hi, lo;
      split2<T>(v[0] * s, v[1] * s, hi.x, lo.x);
      split2<T>(v[2] * s, v[3] * s, hi.y, lo.y);
      split2<T>(v[4] * s, v[5] * s, hi.z, lo.z);
      split2<T>(v[6] * s, v[7] * s, hi.w, lo.w);
      // columns [0, R) of the panels hold the first parts, [R, 2R) the second
      const int ch = lane8, cl = G + lane8;
      const uint32_t at_hi = (ch >> 3) * S::ROWS + swizzled(r, ch & 7), at_lo = (cl >> 3) * S::ROWS + swizzled(r, cl & 7);
      for (int i = 0; i < C; ++i) {
        const int q = (crank + i) % C;
        unsigned char* to = q != crank ? cluster.map_shared_rank(panels, q) : panels;
        *reinterpret_cast<uint4*>(to + at_hi) = hi;
        *reinterpret_cast<uint4*>(to + at_lo) = lo;
        if (SCALED && lane8 == 0) *(q != crank ? cluster.map_shared_rank(&back[r], q) : &back[r]) = b;
      }
    }
  }
  if (C > 1)
    cluster.sync();  // (the last access to another CTA's shared memory lies before)
  else
    __syncthreads();

  // ---- out = base + hidden up, 64 columns a stage ----
  // Four warps have the even stages, four the odd ones: a stage's chain (products,
  // sums, base, stores) takes about a microsecond, which one after the other would
  // bound the kernel.  A warp copies and stores the 32 rows that it adds to.
  const T* up = static_cast<const T*>(a.second) + (int64_t)group * a.rank * N;
  if (issuer) {
    if (lane == 0) {
      tc_fence_after();
      fence_async_cluster();  // (the panels that all CTAs have written)
      for (int i = 0; i < nb; ++i) {
        if (!wait.alone(&in2[i % ST], (i / ST) & 1)) break;
        if (i >= SUMS && !wait.alone(&drained[i % SUMS], (i / SUMS - 1) & 1)) break;
        tc_fence_after();
        fence_async_shared();
        const uint32_t b = ring_at + (i % ST) * S::STAGE + S::ROWS;
#pragma unroll
        for (int k = 0; k < 2 * R / 16; ++k)  // 16 columns of the panels, 16 rows of up
          tc_mma_f16(tmem + (i % SUMS) * 64, smem_desc_sw128(panels_at + (k / 4) * S::ROWS + (k % 4) * 32),
                     smem_desc_rows(b + (k % (R / 16)) * 2048), idesc_f16<T>(64, false, true), k > 0);
        tc_commit(&done[i % SUMS]);
      }
    }
    __syncwarp();
  } else {
    const int sub = lane & 7, first = quarter * 32 + (lane >> 3);        // of base and out: rows four apart
    const int up_row = (tid & 127) >> 3, up_chunk = tid & 7;             // rows 16 apart
    const auto fill = [&](int i) {
      const int col = (b0 + i) * 64;
      const uint32_t at = ring_at + (i % ST) * S::STAGE;
      if constexpr (VEC) {
        if (base) {
          const bool in = col + sub * 8 < N;
          const T* from = base + (in ? col + sub * 8 : 0);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (first + 4 * q < count) copy16(at + swizzled(first + 4 * q, sub), from + base_at[first + 4 * q], in);
        }
        const bool in = col + up_chunk * 8 < N;
        const T* from = up + (in ? col + up_chunk * 8 : 0);
#pragma unroll
        for (int r = up_row; r < R; r += 16)
          copy16(at + S::ROWS + swizzled(r, up_chunk), from + (r < a.rank ? r * N : 0), in && r < a.rank);
        copy_arrive(&in2[i % ST]);
      } else {
        const int cb = col + sub * 8, cu = col + up_chunk * 8;
        Loose l[8];
        if (base) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            l[q].load(base + base_at[first + 4 * q] + cb, N - cb, first + 4 * q < count);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            put16(at + swizzled(first + 4 * q, sub),
                  l[q].chunk(Loose::odd(base + base_at[first + 4 * q] + cb), N - cb));
        }
        constexpr int U = R / 16;
#pragma unroll
        for (int q = 0; q < U; ++q) l[q].load(up + (int64_t)(up_row + 16 * q) * N + cu, N - cu, up_row + 16 * q < a.rank);
#pragma unroll
        for (int q = 0; q < U; ++q)
          put16(at + S::ROWS + swizzled(up_row + 16 * q, up_chunk),
                l[q].chunk(Loose::odd(up + (int64_t)(up_row + 16 * q) * N + cu), N - cu));
        mbar_arrive(&in2[i % ST]);
      }
    };
    for (int i = half; i < min(ST, nb); i += 2) fill(i);
    const float bk = back[mine];
    for (int j = half; j < nb; j += 2) {
      const int col = (b0 + j) * 64;
      unsigned char* tile = ring + (j % ST) * S::STAGE;
      // (the rows of base; products follow them)
      if (lost || !wait.warp(&in2[j % ST], (j / ST) & 1) || !wait.warp(&done[j % SUMS], (j / SUMS) & 1)) {
        for (; j < nb; j += 2)
          for (int r = quarter * 32; r < min(quarter * 32 + 32, count); ++r)
            for (int c = (b0 + j) * 64 + lane; c < min((b0 + j) * 64 + 64, N); c += 32) out[out_at[r] + c] = from_f32<T>(NAN);
        break;
      }
      if (quarter * 32 >= count) {  // (no rows here: only the copies of up)
        if (lane == 0) mbar_arrive(&drained[j % SUMS]);
        if (j + ST < nb) fill(j + ST);
        continue;
      }
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[32];
        tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + (j % SUMS) * 64 + h * 32, v);
        uint4 y[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          y[c] = base ? *reinterpret_cast<const uint4*>(tile + swizzled(mine, h * 4 + c)) : make_uint4(0, 0, 0, 0);
        tmem_ld_wait();
        if (h == 1) {
          tc_fence_before();
          if (lane == 0) mbar_arrive(&drained[j % SUMS]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t w[4] = {y[c].x, y[c].y, y[c].z, y[c].w};
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2(w[e], T());
            o[e] = pack2(fmaf(v[c * 8 + 2 * e], bk, f.x), fmaf(v[c * 8 + 2 * e + 1], bk, f.y), T());
          }
          *reinterpret_cast<uint4*>(tile + swizzled(mine, h * 4 + c)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      __syncwarp();
      if constexpr (VEC) {
        uint4 o[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] = *reinterpret_cast<const uint4*>(tile + swizzled(first + 4 * q, sub));
        if (col + sub * 8 < N) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (first + 4 * q < count)
              *reinterpret_cast<uint4*>(out + out_at[first + 4 * q] + col + sub * 8) = o[q];
        }
      } else {
        // a row's 64 columns, two elements a lane
        const unsigned char* from = tile + (lane & 7) * 2;
#pragma unroll 4
        for (int r = quarter * 32; r < min(quarter * 32 + 32, count); ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c = col + h * 32 + lane;
            const uint16_t v = *reinterpret_cast<const uint16_t*>(from + swizzled(r, h * 4 + (lane >> 3)));
            if (c < N) reinterpret_cast<uint16_t*>(out)[out_at[r] + c] = v;
          }
      }
      // The slot's next stage, whoever will add to it: its rows of this warp have
      // been read by this warp, its products are done.
      __syncwarp();
      if (j + ST < nb) fill(j + ST);
    }
    copy_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (gave_up) wait.settle(&last, lost ? 1 : 0, issuer && lane == 0);
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, SUMS * 64);
  }
}

template <typename T, int R, bool VEC>
cudaError_t launch_tensor_one(const AdapterArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const auto kernel = adapter_tensor_kernel<T, R, VEC>;
  const cudaError_t e = raise_shared(kernel, TensorShared<R>::BYTES, done);
  if (e != cudaSuccess) return e;
  return launch_clustered(kernel, a, TENSOR_THREADS, TensorShared<R>::BYTES, true, s);
}

template <typename T>
cudaError_t launch_tensor(const AdapterArgs& a, bool vec, cudaStream_t s) {
  if (a.rank <= 16) return vec ? launch_tensor_one<T, 16, true>(a, s) : launch_tensor_one<T, 16, false>(a, s);
  if (a.rank <= 32) return vec ? launch_tensor_one<T, 32, true>(a, s) : launch_tensor_one<T, 32, false>(a, s);
  if (a.rank <= 64) return vec ? launch_tensor_one<T, 64, true>(a, s) : launch_tensor_one<T, 64, false>(a, s);
  return vec ? launch_tensor_one<T, 128, true>(a, s) : launch_tensor_one<T, 128, false>(a, s);
}

}  // namespace moe
