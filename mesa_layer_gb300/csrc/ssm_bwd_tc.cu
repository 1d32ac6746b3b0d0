// ssm_bwd_tc.cu -- the selective scan's gradients on the tensor cores (bf16, dk = 128 and dv 64 or 128, or both
// 64; formulas in ssm_bwd.cu, operand formats in ssm_tc.cuh).
//
// Two walks over the chunks (mesa_ssm_chain_tc_kernel) leave the states before and the adjoints after every chunk as
// bf16 operands S^T, R^T [dk][dv]; then every chunk's gradients come from its rows and these two, chunk by chunk:
//     Q K^T, g V^T -> M' = (Q K^T) o E, W = (g V^T) o E D;    dQ = f (g S) + W K,   dK = c D (V R) + W^T Q,
//     du = c (K R^T) + M'^T g,   dV = D du + skip g.
// Eight products of 128^3 a chunk (P = 128).  The scales f, c D and c are put on where the products lie in tensor memory,
// with the sums that the decays' gradients need on the way.  The pairs' terms X = (Q K^T) o W stay fp32.  A token's sum over
// readers i >= t and writers j < t is put together from terms that belong to it alone, by blocks of 32 tokens: those of its
// own block (writers' running sums, added over the readers), its block's readers with earlier blocks' writers, its block's
// writers with later blocks' readers, and whole blocks on either side.  (Run along the chunk as F(t + 1) = F(t) - sum_j X_tj +
// sum_i X_it, 2^-24 of a loud document stayed in the next one: 0.1 of ddt where the first was 1e6 times as loud.)
// du . v is the sum of the same terms (X / D over a token's readers) and c (V R) . k, not a product with du: M's rounding
// to bf16 would be in it (ddt 1.6e-3 off before its own rounding, so 3e-4; the sum of ddt over a head 3.7e-3, so 7e-4).
#include "launch.h"
#include "ssm_tc.cuh"

namespace mesa {

using namespace ssm;

namespace {

// shared memory: Q | K | V | G | R | S (dv = 128: then W) | [W] | M' | misc
template <int P>
struct Grad {
  static constexpr uint32_t K = QK_TILE, V = 2 * QK_TILE, G = V + V_TILE<P>, R = G + V_TILE<P>, S = R + V_TILE<P>,
                            W = P == 128 ? S : S + V_TILE<P>, M = W + QK_TILE, MISC = M + QK_TILE;
};
struct GradMisc {
  alignas(16) float rec[REC];  // the chunk's gates; once every block is done, by rows' warp and token: its rows' sum of X / D
  float frob[2][16];
  float scan[4][4];  // sums over a warp's tokens: of what it reads from before warp 0, 1, 2; of what it writes past the chunk
  uint64_t full1, full2, c1, c2, e, fg, h, a_done, b_done, c_done, f_done, qk_staged, v_staged, drain;
  uint32_t tmem;
  int gave_up;
  int odd;  // something of a token of the chunk's is not finite
};
// Marks of chunks that hold what is not finite, by column, in the gates' place once these have been read: the first such row of
// K, the last of Q and of G plus one (they reach the gradients from there on, or up to there).
constexpr int MARK_K = 0, MARK_Q = DK, MARK_G = 2 * DK, MARKS = R_START;
static_assert(MARK_G + 128 <= (REC - MARKS) * 4, "the gates' part that the columns' sums leave");
template <int P>
constexpr uint32_t kGradSmem = Grad<P>::MISC + sizeof(GradMisc);
static_assert(kGradSmem<128> <= 232448, "shared memory per block");
// Tensor memory: Q K^T, then du | g V^T, then the diagonal blocks' pairs and sums by token | dQ | dK.  The sums' columns (T_SUM:
// of the block beside the token's own), by quarter of the channels (X_ROW: of the chunk's tokens; the token's own quarter holds
// its own block's share of its sum over readers and writers):
constexpr uint32_t T_A = 0, T_B = 128, T_DQ = 256, T_DK = 384;
__device__ __forceinline__ uint32_t T_SUM(int w) { return T_B + 32 * ((w + 1) & 3); }
constexpr int X_ROW = 0, X_IN = 4, X_OUT = 8, X_GV = 12, X_DIAG = 13;

__device__ __forceinline__ void tmem_put(uint32_t taddr, float x) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};\n" ::"r"(taddr), "r"(__float_as_uint(x)) : "memory");
}
// The sum over the warp's lanes of x[lane % 8].
__device__ __forceinline__ float transposed_sum(float (&x)[8], int lane) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; i++) {
      const float give = up ? x[i] : x[i + o], keep = up ? x[i + o] : x[i];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  float y = x[0];
  y += __shfl_xor_sync(0xffffffffu, y, 8);
  return y + __shfl_xor_sync(0xffffffffu, y, 16);
}
// What is not finite in one token's row meets the zeros of the tokens that it has nothing to do with, in W K, W^T Q and M'^T g
// (ssm_tc.cuh).  By a whole warp, in chunks that have any: what is not finite in the rows of K, Q and G goes to marks and is
// taken out of the tiles, and M' and W get their zeros above the diagonal (formed as 0 times what is not finite, they are not).
template <int P>
__device__ __noinline__ void take_out(uint8_t *sm, uint8_t *marks, int lane) {
  using O = Grad<P>;
  const int c = lane & 15;  // half a warp a tile, a lane eight columns
#pragma unroll 1
  for (int i = lane >> 4; i < 3; i += 2) {
    uint8_t *tile = sm + (i == 0 ? O::K : i == 1 ? 0 : O::G), *to = marks + (i == 0 ? MARK_K : i == 1 ? MARK_Q : MARK_G) + 8 * c;
    if (i == 2 && 8 * c >= P) break;
    for (int e = 0; e < 8; e++) to[e] = i == 0 ? kNoRow : 0;
#pragma unroll 1
    for (int t = 0; t < L; t++) {
      uint4 *at = reinterpret_cast<uint4 *>(tile + tile_off(t, c, L));
      if (!odd_words(*at)) continue;
      uint16_t *x = reinterpret_cast<uint16_t *>(at);
      for (int e = 0; e < 8; e++)
        if (odd_word(x[e])) {
          x[e] = 0;
          to[e] = (uint8_t)(i == 0 ? min((int)to[e], t) : t + 1);
        }
    }
  }
#pragma unroll 1
  for (int t = lane >> 4; t < L; t += 2)
#pragma unroll 1
    for (int e = max(t + 1 - 8 * c, 0); e < 8; e++) *word_at(sm + O::M, t, 8 * c + e) = *word_at(sm + O::W, t, 8 * c + e) = 0;
  tc::fence_smem_to_async();
  __syncwarp();
}
// NaN in the gradients of row t that marks say (from where they leave, or in the heads' parts in memory); whether there is any.
// (Calls, so that the usual chunk's code stays as short as without.)
__device__ __noinline__ bool spoil_qk(uint8_t *q, uint8_t *k, const uint8_t *marks, int t, int n0, float *dq, float *dk) {
  bool any = false;
  for (int n = n0; n < n0 + 32; n++) {
    const bool a = marks[MARK_K + n] <= t, b = marks[MARK_Q + n] > t;
    any |= a || b;
    if (a) *word_at(q, t, n) = 0x7fff;
    if (b) *word_at(k, t, n) = 0x7fff;
    if (a && dq) dq[n] = NAN;
    if (b && dk) dk[n] = NAN;
  }
  return any;
}
__device__ __noinline__ bool spoil_v(uint8_t *v, const uint8_t *marks, int t, int p0, int n) {
  bool any = false;
  for (int p = p0; p < p0 + n; p++)
    if (marks[MARK_G + p] > t) any = true, *word_at(v, t, p) = 0x7fff;
  return any;
}
// L2 prefetches of what the next chunk's copies will read.
__device__ __forceinline__ void prefetch_tile(const void *map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];\n" ::"l"(map), "r"(x), "r"(y), "r"(z) : "memory");
}
__device__ __forceinline__ void prefetch_bytes(const void *p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(p), "r"(bytes) : "memory");
}

// A resident CTA per SM over `chunks` chunks of all units, 576 threads: warps 0-15 (lane quarter warp % 4, column
// quarter warp / 4), 16 products, 17 copies.
template <int N, int P>
__global__ void __launch_bounds__(576, 1)
    mesa_ssm_grads_tc_kernel(SsmArgs a, int NC, int chunks, const float *records, const uint8_t *states, const uint8_t *adjoints,
                             float *sums, float *dqp, float *dkp, const __grid_constant__ CUtensorMap mapQ,
                             const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                             const __grid_constant__ CUtensorMap mapG, const __grid_constant__ CUtensorMap mapDq,
                             const __grid_constant__ CUtensorMap mapDk, const __grid_constant__ CUtensorMap mapDv) {
  using O = Grad<P>;
  extern __shared__ __align__(1024) uint8_t sm[];
  if (tc::smem_u32(sm) & 1023) {  // (swizzled tiles need it; the declaration asks for it)
    ahead_done();
    if (threadIdx.x == 0) atomicOr(a.status, tc::kErrMmaTimeout);
    return;
  }
  GradMisc *m = reinterpret_cast<GradMisc *>(sm + O::MISC);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;  // (warp: uniform)
  auto bar = [](uint64_t &b) { return tc::smem_u32(&b); };
  volatile int *gave_up = &m->gave_up;
  const unsigned limit = a.wait_limit;
  if (N < DK) clear_halves(sm, 2);
  if (warp == 16) tc::tmem_alloc(tc::smem_u32(&m->tmem), 512);
  if (tid == 544) {
    for (uint64_t *b : {&m->full1, &m->full2, &m->c1, &m->c2, &m->e, &m->fg, &m->h, &m->drain}) tc::mbar_init(bar(*b), 1);
    for (uint64_t *b : {&m->a_done, &m->b_done, &m->c_done, &m->qk_staged, &m->v_staged}) tc::mbar_init(bar(*b), 16);
    tc::mbar_init(bar(m->f_done), 4);
    m->gave_up = m->odd = 0;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = __shfl_sync(0xffffffffu, m->tmem, 0);
  uint8_t *const marks = reinterpret_cast<uint8_t *>(m->rec + MARKS);
  auto odd = [&]() { return *static_cast<volatile int *>(&m->odd) != 0; };
  auto warp_arrive = [&](uint64_t &b) {  // one arrival per warp, after what its lanes did
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };
  bool ok = true;
  auto need = [&](uint64_t &b, uint32_t parity) {  // a warp's wait; once a lane has given up, the warp has
    ok = __all_sync(0xffffffffu, ok && wait(bar(b), parity, limit, gave_up));
    tc::fence_after_sync();
    return ok;
  };
  int sent1 = 0, sent2 = 0;  // chunks asked for (warp 17)

  may_follow();
  if (warp != 17) ahead_done();
  if (warp < 16) {
    const int w = warp & 3, b = warp >> 2, t = 32 * w + lane;  // row t, columns of quarter b
    const uint32_t tl = tbase + ((uint32_t)(32 * w) << 16);
    uint32_t bad = 0;
    // What the steps' gradients of a chunk need (one warp for each 32 tokens: not the diagonal block's, which takes longest).
    // They are put together while the next chunk's products run.
    const bool teller = b == ((w + 1) & 3);
    struct Steps {
      float in, from0, from1, from2;  // what the token reads from before the chunk, from the blocks 0, 1, 2 before its own
      float own, out, past;  // its own block's pairs and what crosses the whole chunk; what it writes for later blocks, past the chunk
      float duv, gv, raw, step;
      int at, start;
    } last;
    last.at = -1;
    auto steps = [&]() {
      const int u = last.at / NC, c = last.at - u * NC, h = u % a.H;
      const bool in = c * L + t < a.T;
      const float reads0 = last.in, reads1 = reads0 + last.from0, reads2 = reads1 + last.from1;
      float suf = reads2 + last.from2, pre = last.out + last.past;  // over the warp: readers from t on, writers before t
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float p = __shfl_down_sync(0xffffffffu, suf, o), q = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane + o < 32) suf += p;
        if (lane >= o) pre += q;
      }
      pre = __shfl_up_sync(0xffffffffu, pre, 1);
      if (lane == 0) pre = 0.0f;
      const float s0 = warp_sum(reads0), s1 = warp_sum(reads1), s2 = warp_sum(reads2), s3 = warp_sum(last.past);
      if (lane == 0) m->scan[0][w] = s0, m->scan[1][w] = s1, m->scan[2][w] = s2, m->scan[3][w] = s3;
      group_or(2, 128, false);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        if (i > w) suf += m->scan[w < 3 ? w : 0][i];
        if (i < w) pre += m->scan[3][i];
      }
      const float da = last.start == t ? 0.0f : (last.own + pre) + suf;
      const float dd = in ? fmaf(a.A[h], da, last.duv) * sigmoid(last.raw) : 0.0f;
      if (in) {
        if (!isfinite(dd)) bad = 0x7f80u;
        const size_t i = (size_t)u * a.T + c * L + t;
        if (a.gates_f32)
          static_cast<float *>(a.ddt)[i] = dd;
        else
          static_cast<__nv_bfloat16 *>(a.ddt)[i] = __float2bfloat16_rn(dd);
      }
      const float sA = warp_sum(in ? last.step * da : 0.0f), sb = warp_sum(dd), sg = warp_sum(last.gv);
      if (lane == 0) {  // a warp's tokens each
        const size_t n = (size_t)chunks * 4, i = (size_t)last.at * 4 + w;
        sums[i] = sA;
        sums[n + i] = sb;
        sums[2 * n + i] = sg;
      }
    };
    for (int at = blockIdx.x, it = 0; at < chunks; at += gridDim.x, it++) {
      const uint32_t par = it & 1;
      const int u = at / NC, c = at - u * NC, h = u % a.H;
      const bool in = c * L + t < a.T;
      const float raw = in ? a.dt[(size_t)u * a.T + c * L + t] + (a.dt_bias ? a.dt_bias[h] : 0.0f) : 0.0f;
      // <S, R>: 8 P bytes a thread of each
      need(m->full2, par);  // (a warp that gives up goes on to the next barrier with the others)
      const float *r = m->rec;
      const float r_in = r[R_IN + t], step = r[R_STEP + t], f = r_in * r[R_FIRST + w], ct = r[R_OUT + t] * r[R_LAST + w],
                  mine = r[R_LOG + t], mine_lo = lo_of(r, t), across = r[R_ALL];
      const int start = start_of(r, t);
      {
        u64 x2 = 0;
#pragma unroll 2
        for (int i = tid; i < (int)(V_TILE<P> / 16); i += 512) {
          const uint4 x = *reinterpret_cast<const uint4 *>(sm + O::S + 16 * i), y = *reinterpret_cast<const uint4 *>(sm + O::R + 16 * i);
          x2 = fma2(of_bf2(x.x), of_bf2(y.x), x2);
          x2 = fma2(of_bf2(x.y), of_bf2(y.y), x2);
          x2 = fma2(of_bf2(x.z), of_bf2(y.z), x2);
          x2 = fma2(of_bf2(x.w), of_bf2(y.w), x2);
        }
        const float x = warp_sum(sum2(x2));
        if (lane == 0) m->frob[par][warp] = x;
      }
      if (group_or(1, 512, !ok)) {  // (S has been read: W may take its place)
        ok = false;
        break;
      }
      // ---- M', W and the pairs' sums: block (w, b), eight columns at a time ----
      if (teller && it > 0) steps();
      float row = 0.0f, gv = 0.0f, diag = 0.0f, col = 0.0f;  // col: column 32 b + lane
      need(m->c1, par);
      if (b <= w) {
        const float fac = b < w ? r[R_BETWEEN + 4 * w + b] * r_in : 1.0f;
        const u64 fac2 = pack2(fac, fac);
        u64 row2 = 0;
        const uint32_t on = b < w ? 0xffffffffu : (0xffffffffu >> (31 - lane)) & (0xffffffffu << max(start - 32 * w, 0));  // columns that count
        const float *rj = r + (b < w ? R_OUT : R_LOG) + 32 * b, *sj = r + R_STEP + 32 * b;
        const uint32_t *lo_pairs = reinterpret_cast<const uint32_t *>(r + R_LO) + 16 * b;
        const u64 mine2 = pack2(mine, mine), lo2 = pack2(mine_lo, mine_lo);
        float x[2][8], y[2][8];
        tc::tmem_ld8(tl + T_A + 32 * b, x[0]);
        tc::tmem_ld8(tl + T_B + 32 * b, y[0]);
        auto piece = [&](int cc, float (&x)[8], float (&y)[8]) {
          uint32_t om[4], ow[4];
#pragma unroll
          for (int q = 0; q < 2; q++) {
            const ulonglong2 rv = *reinterpret_cast<const ulonglong2 *>(rj + 8 * cc + 4 * q),
                             sv = *reinterpret_cast<const ulonglong2 *>(sj + 8 * cc + 4 * q);
#pragma unroll
            for (int i = 0; i < 2; i++) {
              const int j = 4 * q + 2 * i;
              const u64 se = i ? sv.y : sv.x, x2 = pack2(x[j], x[j + 1]), y2 = pack2(y[j], y[j + 1]);
              u64 e = i ? rv.y : rv.x;
              if (b < w) {
                e = mul2(fac2, e);
              } else {  // the diagonal block: e = 0 where a column does not count
                float l0, l1;
                unpack2(add2(sub2(mine2, e), sub2(lo2, of_bf2(lo_pairs[4 * cc + 2 * q + i]))), l0, l1);
                e = pack2(on >> (8 * cc + j) & 1 ? rule::ex2(l0) : 0.0f, on >> (8 * cc + j + 1) & 1 ? rule::ex2(l1) : 0.0f);
              }
              const u64 m2 = mul2(x2, e);
              u64 z2 = mul2(m2, y2);
              om[2 * q + i] = bf2(m2);
              ow[2 * q + i] = bf2(mul2(y2, mul2(e, se)));
              if (b == w) {
                float z0, z1;
                unpack2(z2, z0, z1);
                if (8 * cc + j == lane) gv = y[j], diag = z0, z0 = 0.0f;
                if (8 * cc + j + 1 == lane) gv = y[j + 1], diag = z1, z1 = 0.0f;
                z2 = pack2(z0, z1);
              }
              row2 = fma2(z2, se, row2);
              unpack2(z2, x[j], x[j + 1]);
            }
          }
          const uint32_t to = tile_off(t, 4 * b + cc, L);
          *reinterpret_cast<uint4 *>(sm + O::M + to) = make_uint4(om[0], om[1], om[2], om[3]);
          *reinterpret_cast<uint4 *>(sm + O::W + to) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
          if (b == w) {  // (for later, in g V^T's place, which has been read)
            tc::tmem_st8(tl + T_B + 32 * b + 8 * cc, x);
          } else {
            const float sum = transposed_sum(x, lane);
            if (lane >> 3 == cc) col = sum;
          }
        };
#pragma unroll 1
        for (int cc = 0; cc < 4; cc += 2) {
          tc::tmem_ld_wait();
          tc::tmem_ld8(tl + T_A + 32 * b + 8 * cc + 8, x[1]);
          tc::tmem_ld8(tl + T_B + 32 * b + 8 * cc + 8, y[1]);
          piece(cc, x[0], y[0]);
          tc::tmem_ld_wait();
          if (cc == 0) {
            tc::tmem_ld8(tl + T_A + 32 * b + 16, x[0]);
            tc::tmem_ld8(tl + T_B + 32 * b + 16, y[0]);
          }
          piece(cc + 1, x[1], y[1]);
        }
        row = sum2(row2);
        if (b == w && !isfinite(diag * step)) m->odd = 1;  // ((q . k) (g . v) D: something of this row's is not)
      } else {
#pragma unroll
        for (int cc = 0; cc < 4; cc++) {
          const uint32_t to = tile_off(t, 4 * b + cc, L);
          *reinterpret_cast<uint4 *>(sm + O::M + to) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4 *>(sm + O::W + to) = make_uint4(0, 0, 0, 0);
        }
      }
      tc::fence_smem_to_async();
      tc::fence_before_sync();
      warp_arrive(m->a_done);
      // ---- f (g S) and c D (V R), with what passes into and out of the chunk ----
      need(m->c2, par);
      auto scaled = [&](uint32_t col, const uint8_t *tile, float s) {  // returns the row's product with the tile's, unscaled
        const u64 s2 = pack2(s, s);
        u64 dot = 0;
        if (32 * b >= N) return 0.0f;  // (no such channels)
#pragma unroll
        for (int hh = 0; hh < 2; hh++) {
          float x[16];
          tc::tmem_ld16(tl + col + 32 * b + 16 * hh, x);
          uint4 q[2];
#pragma unroll
          for (int k = 0; k < 2; k++) q[k] = *reinterpret_cast<const uint4 *>(tile + tile_off(t, 4 * b + 2 * hh + k, L));
          tc::tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 2; k++) {
            const uint32_t qs[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
              const int e = 8 * k + 2 * i;
              const u64 y = pack2(x[e], x[e + 1]);
              dot = fma2(y, of_bf2(qs[i]), dot);
              unpack2(mul2(y, s2), x[e], x[e + 1]);
            }
          }
          tc::tmem_st16(tl + col + 32 * b + 16 * hh, x);
        }
        return sum2(dot);
      };
      const float x_in = f * scaled(T_DQ, sm, f), x_out = ct * scaled(T_DK, sm + O::K, ct * step);
      tc::tmem_st_wait();
      tc::fence_before_sync();
      warp_arrive(m->b_done);
      // ---- the diagonal block's sums: its columns', and of the pairs with readers from token 32 w + lane on and writers before
      // it (off the products' way) ----
      if (b == w) {
        float run = 0.0f;  // of this lane's row
#pragma unroll 1
        for (int cc = 0; cc < 4; cc++) {
          float x[8], y[8];  // X / D; its steps' multiples summed along the row so far
          tc::tmem_ld8(tl + T_B + 32 * b + 8 * cc, x);
          tc::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; j++) {
            const bool on = lane >= 8 * cc + j;  // (above the diagonal: 0 times what may not be finite)
            if (!on) x[j] = 0.0f;
            y[j] = on ? run : 0.0f;
            run = fmaf(x[j], __shfl_sync(0xffffffffu, step, 8 * cc + j), run);
          }
          const float pairs = transposed_sum(y, lane), sum = transposed_sum(x, lane);
          if (lane >> 3 == cc) row = pairs, col = sum;
        }
      }
      // ---- c (K R^T); the sums so far ----
      need(m->e, par);
      {
        constexpr int V = P / 4;
        float x[V];
        tc::tmem_ld<V>(tl + T_A + V * b, x);
        tc::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < V; i++) x[i] *= ct;
        tc::tmem_st<V>(tl + T_A + V * b, x);
        if (b <= w) m->rec[w * L + 32 * b + lane] = col;  // (every block is done: the gates have been read)
        tmem_put(tl + T_SUM(w) + X_ROW + b, row);
        tmem_put(tl + T_SUM(w) + X_IN + b, x_in);
        tmem_put(tl + T_SUM(w) + X_OUT + b, x_out);
        if (b == w) tmem_put(tl + T_SUM(w) + X_GV, gv), tmem_put(tl + T_SUM(w) + X_DIAG, diag);
        tc::tmem_st_wait();
        tc::fence_before_sync();
        warp_arrive(m->c_done);
      }
      // ---- dQ, dK ----
      need(m->fg, par);
      auto put = [&](uint32_t col, uint8_t *tile, float *part) {
        if (32 * b >= N) return;  // (the tiles' second halves stay zero)
        float x[32];
        tc::tmem_ld32(tl + col + 32 * b, x);
        tc::tmem_ld_wait();
#pragma unroll
        for (int cc = 0; cc < 4; cc++) {
          const uint4 o = make_uint4(bf2(x[8 * cc], x[8 * cc + 1]), bf2(x[8 * cc + 2], x[8 * cc + 3]), bf2(x[8 * cc + 4], x[8 * cc + 5]),
                                     bf2(x[8 * cc + 6], x[8 * cc + 7]));
          if (in) bad = rule::absmax_words(bad, o);
          if (!part) {
            *reinterpret_cast<uint4 *>(tile + tile_off(t, 4 * b + cc, L)) = o;
          } else if (in) {
            float4 *dst = reinterpret_cast<float4 *>(part + ((size_t)u * a.T + c * L + t) * N + 32 * b + 8 * cc);
            dst[0] = make_float4(x[8 * cc], x[8 * cc + 1], x[8 * cc + 2], x[8 * cc + 3]);
            dst[1] = make_float4(x[8 * cc + 4], x[8 * cc + 5], x[8 * cc + 6], x[8 * cc + 7]);
          }
        }
      };
      const bool marked = odd();
      put(T_DQ, sm, dqp);
      put(T_DK, sm + O::K, dkp);
      if (marked && 32 * b < N) {
        const size_t row = in ? ((size_t)u * a.T + c * L + t) * N : 0;
        if (spoil_qk(sm, sm + O::K, marks, t, 32 * b, dqp && in ? dqp + row : nullptr, dqp && in ? dkp + row : nullptr) && in) bad = 0x7fff;
      }
      tc::fence_smem_to_async();
      warp_arrive(m->qk_staged);
      // ---- dV ----
      need(m->h, par);
      float later = 0.0f, mine_col = 0.0f;  // X / D over the readers of later blocks, of its own
      if (teller) {  // (all warps' columns are there)
        mine_col = m->rec[w * L + t];
#pragma unroll
        for (int i = 1; i < 4; i++)
          if (i > w) later += m->rec[i * L + t];
      }
      {
        constexpr int V = P / 4;
        const float skip = a.skip ? a.skip[h] : 0.0f;
        const u64 step2 = pack2(step, step), skip2 = pack2(skip, skip);
        float x[V];
        tc::tmem_ld<V>(tl + T_A + V * b, x);
        tc::tmem_ld_wait();
#pragma unroll
        for (int cc = 0; cc < V / 8; cc++) {
          const uint32_t to = tile_off(t, V / 8 * b + cc, L);
          const uint4 g = *reinterpret_cast<const uint4 *>(sm + O::G + to);
          const uint32_t gs[4] = {g.x, g.y, g.z, g.w};
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const u64 du = pack2(x[8 * cc + 2 * i], x[8 * cc + 2 * i + 1]);
            o[i] = bf2(a.skip ? fma2(skip2, of_bf2(gs[i]), mul2(step2, du)) : mul2(step2, du));
          }
          const uint4 y = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4 *>(sm + O::G + to) = y;
          if (in) bad = rule::absmax_words(bad, y);
        }
        if (marked && spoil_v(sm + O::G, marks, t, V * b, V) && in) bad = 0x7fff;
        tc::fence_before_sync();
        tc::fence_smem_to_async();
        warp_arrive(m->v_staged);
      }
      if (group_or(1, 512, !ok)) {
        ok = false;
        break;
      }
      if (tid == 0) m->odd = 0;
      if (!teller) continue;
      tc::fence_after_sync();
      float x[16];
      tc::tmem_ld16(tl + T_SUM(w), x);
      float all = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float4 y = *reinterpret_cast<const float4 *>(&m->frob[par][4 * i]);
        all += (y.x + y.y) + (y.z + y.w);
      }
      tc::tmem_ld_wait();
      tc::fence_before_sync();
      warp_arrive(m->f_done);
      auto four = [&](int i) { return (x[i] + x[i + 1]) + (x[i + 2] + x[i + 3]); };
      const float xo = four(X_OUT);
      last = Steps{four(X_IN), w > 0 ? x[X_ROW] : 0.0f, w > 1 ? x[X_ROW + 1] : 0.0f, w > 2 ? x[X_ROW + 2] : 0.0f,
                   fmaf(across, all, w == 0 ? x[X_ROW] : w == 1 ? x[X_ROW + 1] : w == 2 ? x[X_ROW + 2] : x[X_ROW + 3]), step * later,
                   step * xo, (later + mine_col + x[X_DIAG]) + xo, x[X_GV], raw, step, at, start};
    }
    if (teller && ok && last.at >= 0) steps();
    if (ok && max(bad & 0xffffu, bad >> 16) >= 0x7f80u) atomicOr(a.status, tc::kErrNonFinite);
  } else if (warp == 16) {
    // ---- products ----
    const uint32_t id = idesc_bf16(128, 128, false, false), idB = idesc_bf16(128, 128, false, true),
                   idAB = idesc_bf16(128, 128, true, true), idP = idesc_bf16(128, P, false, true), idPA = idesc_bf16(128, P, true, true);
    auto km = [&](uint32_t where) { return tc::kmajor_desc(tc::smem_u32(sm + where), L, 0); };
    auto mn = [&](uint32_t where) { return tc::mnmajor_desc(tc::smem_u32(sm + where), L, 0); };
    const uint64_t qk = km(0), qm = mn(0), kk = km(O::K), kmn = mn(O::K), vk = km(O::V), gk = km(O::G), gm = mn(O::G), sk = km(O::S),
                   rk = km(O::R), rm = mn(O::R), wk = km(O::W), wm = mn(O::W), mm = mn(O::M);
    for (int at = blockIdx.x, it = 0; at < chunks; at += gridDim.x, it++) {
      const uint32_t par = it & 1;
      if (!need(m->full1, par) || (it > 0 && !need(m->f_done, par ^ 1))) break;
      if (elect_one()) {
#pragma unroll
        for (int s = 0; s < N / 16; s++) tc::mma_f16(tbase + T_A, qk + step128(s), kk + step128(s), id, s > 0);
#pragma unroll
        for (int s = 0; s < P / 16; s++) tc::mma_f16(tbase + T_B, gk + step128(s), vk + step128(s), id, s > 0);
      }
      if (!need(m->full2, par)) break;
      if (elect_one()) {
#pragma unroll
        for (int s = 0; s < P / 16; s++) tc::mma_f16(tbase + T_DQ, gk + step128(s), sk + step128(s), id, s > 0);
        tc::mma_commit(bar(m->c1));
#pragma unroll
        for (int s = 0; s < P / 16; s++) tc::mma_f16(tbase + T_DK, vk + step128(s), rk + step128(s), id, s > 0);
        tc::mma_commit(bar(m->c2));
      }
      if (!need(m->a_done, par)) break;
      if (elect_one()) {
#pragma unroll
        for (int s = 0; s < N / 16; s++) tc::mma_f16(tbase + T_A, kk + step128(s), rm + step_mn(s), idP, s > 0);
        tc::mma_commit(bar(m->e));
      }
      if (!need(m->b_done, par)) break;
      if (odd()) {
        if (!need(m->e, par)) break;  // (K R^T has read K)
        take_out<P>(sm, marks, lane);
      }
      if (elect_one()) {
#pragma unroll
        for (int s = 0; s < 8; s++) tc::mma_f16(tbase + T_DQ, wk + step128(s), kmn + step_mn(s), idB, true);
#pragma unroll
        for (int s = 0; s < 8; s++) tc::mma_f16(tbase + T_DK, wm + step_mn(s), qm + step_mn(s), idAB, true);
        tc::mma_commit(bar(m->fg));
      }
      if (!need(m->c_done, par)) break;
      if (elect_one()) {
#pragma unroll
        for (int s = 0; s < 8; s++) tc::mma_f16(tbase + T_A, mm + step_mn(s), gm + step_mn(s), idPA, true);
        tc::mma_commit(bar(m->h));
      }
    }
  } else if (lane == 0) {
    // ---- copies ----
    // Q and K, V, G arrive at full1, S, R and the gates at full2; the first of each announces them all.
    auto tile = [&](uint32_t where, const CUtensorMap &map, int d, int at, uint64_t &b, int unit_of) {
      const int u = at / NC, y = (at - u * NC) * L, z = unit_of ? a.qk_unit(u) : u;
      for (int i = 0; i < d / 64; i++) tensor_g2s_3d(tc::smem_u32(sm + where) + i * HALF, &map, 64 * i, y, z, bar(b));
    };
    auto fetch_adjoint = [&](int at) {
      tc::mbar_arrive_expect_tx(bar(m->full2), 2 * V_TILE<P> + REC * 4);
      tc::bulk_g2s(tc::smem_u32(sm + O::R), adjoints + (size_t)at * V_TILE<P>, V_TILE<P>, bar(m->full2));
    };
    auto fetch_gates = [&](int at) { tc::bulk_g2s(tc::smem_u32(m->rec), records + (size_t)at * REC, REC * 4, bar(m->full2)); };
    auto fetch_state = [&](int at) {
      tc::bulk_g2s(tc::smem_u32(sm + O::S), states + (size_t)at * V_TILE<P>, V_TILE<P>, bar(m->full2));
    };
    auto fetch_v = [&](int at) {
      tc::mbar_arrive_expect_tx(bar(m->full1), 2 * L * N * 2 + 2 * V_TILE<P>);
      tile(O::V, mapV, P, at, m->full1, 0);
    };
    auto fetch_qk = [&](int at) {
      tile(0, mapQ, N, at, m->full1, 1);
      tile(O::K, mapK, N, at, m->full1, 1);
    };
    auto fetch_g = [&](int at) { tile(O::G, mapG, P, at, m->full1, 0); };
    auto prefetch = [&](int at) {
      const int u = at / NC, y = (at - u * NC) * L, uk = a.qk_unit(u);
#pragma unroll
      for (int i = 0; i < N / 64; i++) prefetch_tile(&mapQ, 64 * i, y, uk), prefetch_tile(&mapK, 64 * i, y, uk);
#pragma unroll
      for (int i = 0; i < P / 64; i++) prefetch_tile(&mapV, 64 * i, y, u), prefetch_tile(&mapG, 64 * i, y, u);
      prefetch_bytes(states + (size_t)at * V_TILE<P>, V_TILE<P>);
      prefetch_bytes(adjoints + (size_t)at * V_TILE<P>, V_TILE<P>);
      prefetch_bytes(records + (size_t)at * REC, REC * 4);
    };
    if ((int)blockIdx.x < chunks) {
      const int at = blockIdx.x;
      fetch_v(at);
      fetch_qk(at);
      fetch_g(at);
      ahead_done();  // (the states, adjoints and gates; the rows are the call's inputs)
      fetch_adjoint(at);
      fetch_state(at);
      fetch_gates(at);
      sent1 = sent2 = 1;
    }
    // (Each as soon as nothing reads it: V after the first products, R after K R^T, S or W after dQ and dK's products,
    // Q, K and G after the gradients have left from there, the gates after the columns' sums.)
    for (int at = blockIdx.x, it = 0; at < chunks; at += gridDim.x, it++) {
      const uint32_t par = it & 1;
      const int u = at / NC, y = (at - u * NC) * L, uk = a.qk_unit(u), next = at + gridDim.x;
      const bool more = next < chunks;
      if (more) prefetch(next);
      if (!(ok = wait(bar(m->c2), par, limit, gave_up))) break;
      if (more) {  // (what is announced is sent, whatever happens)
        fetch_v(next);
        sent1++;
      }
      ok = wait(bar(m->e), par, limit, gave_up);
      if (more) {
        fetch_adjoint(next);
        sent2++;
      }
      ok = ok && wait(bar(m->fg), par, limit, gave_up);
      if (more) fetch_state(next);
      ok = ok && wait(bar(m->qk_staged), par, limit, gave_up);
      if (!dqp && ok) {
#pragma unroll
        for (int i = 0; i < N / 64; i++) {
          tensor_s2g_3d(&mapDq, tc::smem_u32(sm) + i * HALF, 64 * i, y, uk);
          tensor_s2g_3d(&mapDk, tc::smem_u32(sm + O::K) + i * HALF, 64 * i, y, uk);
        }
        tc::bulk_commit();
      }
      if (more) {
        tc::bulk_wait_read();
        fetch_qk(next);
      }
      ok = ok && wait(bar(m->v_staged), par, limit, gave_up);
      if (more) fetch_gates(next);
      if (ok) {
#pragma unroll
        for (int i = 0; i < P / 64; i++) tensor_s2g_3d(&mapDv, tc::smem_u32(sm + O::G) + i * HALF, 64 * i, y, u);
        tc::bulk_commit();
      }
      if (more) {
        tc::bulk_wait_read();
        fetch_g(next);
      }
      if (!ok) break;
    }
    tc::bulk_wait_all();
  }
  if (!ok) *gave_up = 1;
  __syncthreads();
  // a wait gave up: products and copies still in flight finish before the memory is released
  if (*gave_up) {
    if (warp == 16 && elect_one()) tc::mma_commit(bar(m->drain));
    if (tid == 0) {
      unsigned bits = tc::kErrMmaTimeout;
      if (!tc::mbar_wait(bar(m->drain), 0, tc::kWaitLimit)) bits |= tc::kErrDrainTimeout;
      atomicOr(a.status, bits);
    }
    if (tid == 544 && sent1 > 0 &&
        !(tc::mbar_wait(bar(m->full1), (sent1 - 1) & 1, tc::kWaitLimit) && tc::mbar_wait(bar(m->full2), (sent2 - 1) & 1, tc::kWaitLimit)))
      atomicOr(a.status, tc::kErrDrainTimeout);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 16) tc::tmem_free(tbase, 512);
}

template <int N, int P>
int grads(const SsmArgs &a, const SsmSegments &sg, const SsmTcBwd &ws, cudaStream_t st) {
  CUtensorMap q{}, k{}, v{}, g{}, dq{}, dk{}, dv{};
  const int shared = a.B * a.Hk, NC = (a.T + L - 1) / L, chunks = a.units() * NC, sms = sm_count();
  if (!tmap_units_bf16(&q, a.q, shared, a.T, N) || !tmap_units_bf16(&k, a.k, shared, a.T, N) ||
      !tmap_units_bf16(&v, a.v, a.units(), a.T, P) || !tmap_units_bf16(&g, a.dout, a.units(), a.T, P) ||
      !tmap_units_bf16(&dq, a.dq, shared, a.T, N) || !tmap_units_bf16(&dk, a.dk_out, shared, a.T, N) ||
      !tmap_units_bf16(&dv, a.dv_out, a.units(), a.T, P) || sms <= 0)
    return -1;
  if (cudaFuncSetAttribute(mesa_ssm_grads_tc_kernel<N, P>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGradSmem<P>) != cudaSuccess)
    return -1;
  timing_mark_begin(K_SSM_GRADS, st);
  const bool ok = launch_after(mesa_ssm_grads_tc_kernel<N, P>, chunks < sms ? chunks : sms, 576, kGradSmem<P>, st, a, NC, chunks, sg.records,
                               ws.S, ws.R, ws.sums, ws.dqp, ws.dkp, q, k, v, g, dq, dk, dv);
  timing_mark_end(K_SSM_GRADS, st);
  return ok && cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

// [segments, records | S | R | sums | per-head dq, dk]
size_t parts(const SsmArgs &a, void *workspace, SsmSegments *sg, SsmTcBwd *ws) {
  auto up256 = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t U = a.units(), NC = ((size_t)a.T + L - 1) / L, tiles = U * NC * L * a.dv * 2, part = a.Hk != a.H ? U * a.T * a.dk * 4 : 0;
  size_t at;
  const SsmSegments s = ssm_segments(a.units(), a.T, a.dv, true, workspace, &at);
  if (sg) *sg = s;
  char *base = (char *)workspace;
  at = up256(at);
  const size_t sizes[5] = {tiles, tiles, 3 * U * NC * 4 * sizeof(float), part, part};
  size_t off[5];
  for (int i = 0; i < 5; i++) {
    off[i] = at;
    at += up256(sizes[i]);
  }
  if (ws && workspace)
    *ws = SsmTcBwd{(uint8_t *)base + off[0], (uint8_t *)base + off[1], (float *)(base + off[2]), part ? (float *)(base + off[3]) : nullptr,
                   part ? (float *)(base + off[4]) : nullptr};
  return at;
}

}  // namespace

size_t ssm_tc_backward_workspace(int B, int H, int Hk, int T, int dk, int dv) {
  SsmArgs a{B, H, Hk, T, dk, dv, 1};
  return parts(a, nullptr, nullptr, nullptr);
}

int launch_ssm_backward_tc(const SsmArgs &a, void *workspace, cudaStream_t st) {
  SsmSegments sg;
  SsmTcBwd ws;
  parts(a, workspace, &sg, &ws);
  if (launch_ssm_gates(a, sg, st) != 0 || launch_ssm_chains_tc(a, sg, ws, st) != 0) return -1;
  if ((a.dk == 64 ? grads<64, 64>(a, sg, ws, st) : a.dv == 128 ? grads<128, 128>(a, sg, ws, st) : grads<128, 64>(a, sg, ws, st)) != 0) return -1;
  if (ws.dqp && launch_ssm_group_sum(a, ws.dqp, ws.dkp, st) != 0) return -1;
  return launch_ssm_param_sums(a, ws.sums, 4 * ((a.T + L - 1) / L), st);
}

}  // namespace mesa
