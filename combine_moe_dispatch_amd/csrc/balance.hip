// balance.hip -- the router's balance loss and the router's gradient.
//
// Both walk the logits with one wave per token, the row in registers.  With
// p the token's probabilities, c, n and P a sequence's counts, tokens and
// mean probabilities, the loss is a sum of c P / n, whose gradient needs only
// counts: dl = p (g - <g, p>) with g proportional to c / n^2, times 1 - sigmoid
// for sigmoid scores; the routed weights w add w (gw - <gw, w>) at their ids,
// times the same factor.
//
// Both are streams over the logits (4 T E bytes in, for the gradient as many
// out), so what counts is enough rows in flight: the next token's row is
// loaded before the current one is worked on, rows are 16 bytes a lane where
// E and the pointers allow, and every wave walks a run of neighbouring tokens,
// whose sequence is looked up once and whose counts stay in registers.  65536
// tokens of 256 experts: the gradient 134 MB in 32 to 34 us (4 TB/s; the columns'
// sums 4 us more), where a copy would take 26.  The routed weights come with
// the row (131072 tokens 81 -> 73 us), the gradients go out past the caches
// (73 -> 72).
#include "device_common.h"
#include "experts.h"

namespace moe {

namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;

// Sums and maxima over the wave, the same in every lane: DPP row shifts and
// row broadcasts leave them in lane 63.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float v, float otherwise) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(otherwise), __float_as_int(v),
                                                    CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0x111, 0xf>(v, 0.0f);  // row_shr 1, 2, 4, 8
  v += dpp<0x112, 0xf>(v, 0.0f);
  v += dpp<0x114, 0xf>(v, 0.0f);
  v += dpp<0x118, 0xf>(v, 0.0f);
  v += dpp<0x142, 0xa>(v, 0.0f);  // row_bcast 15, 31
  v += dpp<0x143, 0xc>(v, 0.0f);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp<0x111, 0xf>(v, -INFINITY));
  v = fmaxf(v, dpp<0x112, 0xf>(v, -INFINITY));
  v = fmaxf(v, dpp<0x114, 0xf>(v, -INFINITY));
  v = fmaxf(v, dpp<0x118, 0xf>(v, -INFINITY));
  v = fmaxf(v, dpp<0x142, 0xa>(v, -INFINITY));
  v = fmaxf(v, dpp<0x143, 0xc>(v, -INFINITY));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// A row of E values spread over a wave: VPL of them a lane, VEC neighbours at a
// time (VEC == 4: 16-byte accesses, E % 4 == 0).
template <int VPL, int VEC>
struct Row {
  static __device__ __forceinline__ int expert(int i) {
    return (i / VEC * kWave + lane_id()) * VEC + i % VEC;
  }
  template <class T>
  static __device__ __forceinline__ void load(const T* row, int E, T (&v)[VPL], T absent) {
#pragma unroll
    for (int i = 0; i < VPL; i += VEC) {
      const bool in = expert(i) < E;
      if constexpr (VEC == 4) {
        const int4 q = *reinterpret_cast<const int4*>(row + (in ? expert(i) : 0));
        v[i] = in ? __builtin_bit_cast(T, q.x) : absent;
        v[i + 1] = in ? __builtin_bit_cast(T, q.y) : absent;
        v[i + 2] = in ? __builtin_bit_cast(T, q.z) : absent;
        v[i + 3] = in ? __builtin_bit_cast(T, q.w) : absent;
      } else {
        const T q = row[in ? expert(i) : 0];
        v[i] = in ? q : absent;
      }
    }
  }
  // STREAM: to memory, past the caches
  template <bool STREAM = false>
  static __device__ __forceinline__ void store(float* row, int E, const float (&v)[VPL]) {
#pragma unroll
    for (int i = 0; i < VPL; i += VEC) {
      if (expert(i) >= E) continue;
      if constexpr (VEC == 4) {
        const uint4 q = make_uint4(__float_as_uint(v[i]), __float_as_uint(v[i + 1]),
                                   __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3]));
        if constexpr (STREAM)
          store_stream(reinterpret_cast<uint4*>(row + expert(i)), q);
        else
          *reinterpret_cast<uint4*>(row + expert(i)) = q;
      } else {
        row[expert(i)] = v[i];
      }
    }
  }
};

// LDS hand-off inside one wave.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// From biased logits l (-inf past E) the unnormalised probabilities e and the
// factors r of their gradient (1 - sigmoid; 1 for softmax); returns their
// normaliser 1 / sum.  A sigmoid and its complement come from one exponential
// of -|l|.  Far below zero (all logits under -64) the sigmoids are taken
// relative to the largest, exp(l - top) (1 - sigmoid), so that their sum
// cannot vanish.
template <int VPL>
__device__ __forceinline__ void probabilities(const float (&l)[VPL], int score, float (&e)[VPL],
                                              float (&r)[VPL], float& top) {
  top = l[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) top = fmaxf(top, l[i]);
  top = wave_max(top);
  if (score == 0) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      e[i] = expf(l[i] - top);
      r[i] = 1.0f;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const float t = expf(-fabsf(l[i]));
    const float q = __builtin_amdgcn_rcpf(1.0f + t);  // within an ulp; 1 + t is in [1, 2]
    e[i] = l[i] >= 0.0f ? q : t * q;
    r[i] = l[i] >= 0.0f ? t * q : q;
  }
  if (top < -64.0f) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) e[i] = expf(l[i] - top) * r[i];
  }
}

// The tokens of one wave, one after the other: ids, biased logits and (if
// wanted) routed weights and their gradients of the current one, the next one's
// already on their way.
template <int VPL, int VEC>
struct Tokens {
  using R = Row<VPL, VEC>;
  const float* logits;
  const int32_t* ids;
  const float* weights = nullptr;
  const float* grad_weights = nullptr;
  int E, k, end, step, t;
  float bias[VPL], l[VPL], ahead[VPL];
  int id, id_ahead;
  float w, w_ahead, gw, gw_ahead;

  __device__ __forceinline__ void fetch(int at) {
    if (at >= end) return;
    R::load(logits + (size_t)at * E, E, ahead, -INFINITY);
    const bool slot = lane_id() < k;
    const size_t pair = (size_t)at * k + lane_id();
    id_ahead = slot ? ids[pair] : -1;
    if (grad_weights) {
      w_ahead = slot ? weights[pair] : 0.0f;
      gw_ahead = slot ? grad_weights[pair] : 0.0f;
    }
  }
  __device__ __forceinline__ void init(const float* lg, const float* bs, const int32_t* id_list,
                                       int E_, int k_, int first, int end_, int step_) {
    logits = lg;
    ids = id_list;
    E = E_;
    k = k_;
    end = end_;
    step = step_;
    t = first - step;
    fetch(first);
    if (bs) {
      R::load(bs, E, bias, 0.0f);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) bias[i] = 0.0f;
    }
  }
  // On to the next token; false past the last.
  __device__ __forceinline__ bool next() {
    t += step;
    if (t >= end) return false;
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = ahead[i] + bias[i];
    id = id_ahead;
    w = w_ahead;
    gw = gw_ahead;
    fetch(t + step);
    return true;
  }
  __device__ __forceinline__ bool real() const { return id >= 0 && id < E; }
};

__device__ __forceinline__ int cut(int v, int T) { return min(max(v, 0), T); }
__device__ __forceinline__ int seq_begin(const int32_t* off, int s, int T) {
  return off ? cut(off[s], T) : 0;
}
__device__ __forceinline__ int seq_end(const int32_t* off, int s, int T) {
  return off ? cut(off[s + 1], T) : T;
}

// The first sequence from lo on that ends behind token t (S: none).
__device__ __forceinline__ int sequence_at(const int32_t* off, int lo, int S, int t) {
  if (!off) return 0;
  int hi = S;  // sequences before lo end at or before t, hi is behind it
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (off[mid + 1] <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// The loss.  A block takes a chunk of tokens and goes through the sequences in
// it: its waves add up the probabilities of their tokens in registers, then
// with each other's in LDS.  A sequence inside one chunk is finished there;
// of one that crosses chunks every chunk leaves a part, and the second launch
// adds these up in token order.
// ---------------------------------------------------------------------------
constexpr int kChunks = 1024;     // at most, so that the parts stay few
constexpr int kMinChunk = 16;
// One block for short lists of few sequences, which it takes one after the
// other (64 tokens of 256 experts: 8.3 us against 10.7 by two launches for one
// sequence, 10.8 against 11.1 for 4, 13.4 against 12.7 for 6, 83 against 36 for 64).
constexpr int kOneBlockTokens = 64;
constexpr int kOneBlockSeqs = 4;
constexpr int kOneBlockWaves = 8;
bool one_block(int T, int S) { return T <= kOneBlockTokens && S <= kOneBlockSeqs; }

int chunk_tokens(int T) {
  const int c = (T + kChunks - 1) / kChunks;
  return c < kMinChunk ? kMinChunk : (c + kWaves - 1) / kWaves * kWaves;
}

int chunks_of(int T) {  // one for no tokens too: the first block clears the ticket
  const int chunk = chunk_tokens(T);
  return T == 0 ? 1 : (T + chunk - 1) / chunk;
}

// Parts of the sequence that a chunk begins inside of (0) and of the one that
// it ends inside of, begun in it (1): sums, counts, tokens.
struct Parts {
  float* sums;    // [chunks][2][E]
  int* counts;    // [chunks][2][E]
  int* tokens;    // [chunks][2]
  float* terms;   // [S][expert blocks] of the loss
  unsigned* ticket;
};

__host__ __device__ inline size_t round16(size_t n) { return (n + 15) / 16 * 16; }

size_t parts_bytes(int chunks, int E, int S) {
  const size_t rows = (size_t)chunks * 2;
  return round16(rows * E * 4) * 2 + round16(rows * 4) +
         round16((size_t)S * ((E + kWave - 1) / kWave) * 4) + 16;
}

Parts parts_of(void* ws, int chunks, int E, int S) {
  const size_t rows = (size_t)chunks * 2;
  char* p = static_cast<char*>(ws);
  Parts q;
  q.sums = reinterpret_cast<float*>(p);
  p += round16(rows * E * 4);
  q.counts = reinterpret_cast<int*>(p);
  p += round16(rows * E * 4);
  q.tokens = reinterpret_cast<int*>(p);
  p += round16(rows * 4);
  q.terms = reinterpret_cast<float*>(p);
  p += round16((size_t)S * ((E + kWave - 1) / kWave) * 4);
  q.ticket = reinterpret_cast<unsigned*>(p);
  return q;
}

// Sum over the block in thread order, in thread 0.
template <int WAVES>
__device__ __forceinline__ float block_sum(float v, float (&s)[WAVES]) {
  v = wave_sum(v);
  if (lane_id() == 0) s[threadIdx.x / kWave] = v;
  __syncthreads();
  float total = 0.0f;
  for (int i = 0; i < WAVES; ++i) total += s[i];
  return total;
}

__device__ __forceinline__ float loss_of(const BalanceParams& q, float terms) {
  return terms * ((float)q.E / (float)q.k) * (q.coef / (float)q.S);
}

// ALL: the one block of a short list, which finishes every sequence and the
// loss.
template <int VPL, int VEC, int WAVES, bool ALL>
__global__ void __launch_bounds__(WAVES * kWave)
balance_kernel(BalanceParams q, Parts parts, int chunk) {
  constexpr int kMost = VPL * kWave;
  __shared__ int s_count[kMost];
  __shared__ __align__(16) float s_prob[WAVES][kMost];
  __shared__ int s_tokens[WAVES];
  __shared__ float s_sum[WAVES];
  const int wave = threadIdx.x / kWave;
  const int t0 = ALL ? 0 : blockIdx.x * chunk, t1 = ALL ? q.T : min(q.T, t0 + chunk);
  if (!ALL && blockIdx.x == 0 && threadIdx.x == 0) *parts.ticket = 0;
  float term = 0.0f;
  // the block's next sequence: any, or (empty ones are left to the second
  // launch, however many stand in a row) the first that ends behind token t
  auto following = [&](int s, int t) {
    if (++s < q.S && !ALL && q.seq_offsets[s + 1] <= t)
      s = sequence_at(q.seq_offsets, s, q.S, t);
    return s;
  };
  int end;
  for (int s = ALL ? 0 : sequence_at(q.seq_offsets, 0, q.S, t0); s < q.S; s = following(s, end)) {
    const int begin = seq_begin(q.seq_offsets, s, q.T);
    end = seq_end(q.seq_offsets, s, q.T);
    if (!ALL && begin >= t1) break;
    const int a = max(begin, t0), b = min(end, t1);
    if (!ALL && a >= b) continue;
    for (int e = threadIdx.x; e < q.E; e += WAVES * kWave) s_count[e] = 0;
    __syncthreads();
    float acc[VPL] = {};
    int n = 0;
    Tokens<VPL, VEC> tok;
    tok.init(q.logits, q.bias, q.ids, q.E, q.k, a + wave, b, WAVES);
    while (tok.next()) {
      if (tok.real()) atomicAdd(&s_count[tok.id], 1);
      if (__ballot(tok.real()) == 0) continue;
      ++n;
      float e[VPL], r[VPL], top, sum = 0.0f;
      probabilities<VPL>(tok.l, q.score, e, r, top);
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum += e[i];
      const float inv = 1.0f / wave_sum(sum);
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] = fmaf(e[i], inv, acc[i]);
    }
    Row<VPL, VEC>::store(s_prob[wave], kMost, acc);
    if (lane_id() == 0) s_tokens[wave] = n;
    __syncthreads();
    int tokens = 0;
    for (int i = 0; i < WAVES; ++i) tokens += s_tokens[i];
    const bool whole = ALL || (begin >= t0 && end <= t1);
    const size_t part = (size_t)blockIdx.x * 2 + (begin >= t0 ? 1 : 0);
    for (int e = threadIdx.x; e < q.E; e += WAVES * kWave) {
      float sum = 0.0f;
      for (int i = 0; i < WAVES; ++i) sum += s_prob[i][e];
      const int count = s_count[e];
      if (whole) {
        const float mean = sum / (float)max(tokens, 1);
        q.counts[(size_t)s * q.E + e] = count;
        q.probs[(size_t)s * q.E + e] = mean;
        if (ALL) term += (float)count / (float)max(tokens, 1) * mean;
      } else {
        parts.sums[part * q.E + e] = sum;
        parts.counts[part * q.E + e] = count;
      }
    }
    if (threadIdx.x == 0) *(whole ? &q.tokens[s] : &parts.tokens[part]) = tokens;
    __syncthreads();
  }
  if constexpr (ALL) {
    const float total = block_sum<WAVES>(term, s_sum);
    if (threadIdx.x == 0) q.loss[0] = loss_of(q, total);
  }
}

// Block (expert block, sequence): 16 waves add up the parts of 64 experts.
constexpr int kJoinWaves = 16;

__global__ void __launch_bounds__(kJoinWaves * kWave)
balance_join_kernel(BalanceParams q, Parts parts, int chunk) {
  __shared__ float s_prob[kJoinWaves][kWave];
  __shared__ int s_count[kJoinWaves][kWave], s_tokens[kJoinWaves];
  __shared__ float s_sum[kJoinWaves];
  __shared__ bool s_last;
  const int wave = threadIdx.x / kWave, lane = lane_id();
  for (int s = blockIdx.y; s < q.S; s += gridDim.y) {
    const int begin = seq_begin(q.seq_offsets, s, q.T), end = seq_end(q.seq_offsets, s, q.T);
    const int e = blockIdx.x * kWave + lane;
    const int c0 = begin / chunk, c1 = end > begin ? (end - 1) / chunk : c0;
    float sum = 0.0f;
    int count = 0, n = 0;
    if (c1 > c0 && e < q.E) {
      // a run of chunks to each wave, eight loads on their way at once
      const int per = (c1 - c0 + kJoinWaves) / kJoinWaves;
      const int last = min(c0 + (wave + 1) * per - 1, c1);
#pragma unroll 8
      for (int c = c0 + wave * per; c <= last; ++c) {
        const size_t part = (size_t)c * 2 + (c == c0 ? 1 : 0);
        sum += parts.sums[part * q.E + e];
        count += parts.counts[part * q.E + e];
        n += parts.tokens[part];
      }
    }
    s_prob[wave][lane] = sum;
    s_count[wave][lane] = count;
    if (lane == 0) s_tokens[wave] = n;
    __syncthreads();
    if (wave == 0) {
      float term = 0.0f;
      if (e < q.E) {
        const size_t at = (size_t)s * q.E + e;
        float mean = 0.0f;
        int tokens = 0;
        count = 0;
        if (c1 > c0) {
          for (int i = 0; i < kJoinWaves; ++i) {
            mean += s_prob[i][lane];
            count += s_count[i][lane];
            tokens += s_tokens[i];
          }
          mean /= (float)max(tokens, 1);
        } else if (end > begin) {  // finished by its chunk
          mean = q.probs[at];
          count = q.counts[at];
          tokens = q.tokens[s];
        }
        if (c1 > c0 || end <= begin) {
          q.probs[at] = mean;
          q.counts[at] = count;
          if (e == 0) q.tokens[s] = tokens;
        }
        term = (float)count / (float)max(tokens, 1) * mean;
      }
      term = wave_sum(term);
      if (lane == 0) parts.terms[(size_t)s * gridDim.x + blockIdx.x] = term;
    }
    __syncthreads();
  }
  // the block that is done last adds up the terms, in their order
  if (threadIdx.x == 0)
    s_last = __hip_atomic_fetch_add(parts.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
             gridDim.x * gridDim.y - 1;
  __syncthreads();
  if (!s_last) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  float sum = 0.0f;
  for (size_t i = threadIdx.x; i < (size_t)q.S * gridDim.x; i += kJoinWaves * kWave)
    sum += parts.terms[i];
  const float total = block_sum<kJoinWaves>(sum, s_sum);
  if (threadIdx.x == 0) q.loss[0] = loss_of(q, total);
}

// ---------------------------------------------------------------------------
// The gradient.  A wave's tokens are neighbours; with BIAS it also adds up its
// rows, and the block leaves their sum for the second launch.
// ---------------------------------------------------------------------------
constexpr int kGradBlocks = 1024;

template <int VPL, int VEC, bool BIAS>
__global__ void __launch_bounds__(kThreads)
route_grad_kernel(RouteGradParams q, int per_wave) {
  using R = Row<VPL, VEC>;
  __shared__ __align__(16) float s_row[kWaves][VPL * kWave];  // routed gradients, then sums
  const int wave = threadIdx.x / kWave, lane = lane_id();
  const int64_t first = ((int64_t)blockIdx.x * kWaves + wave) * per_wave;
  const int t0 = (int)min(first, (int64_t)q.T), t1 = (int)min(first + per_wave, (int64_t)q.T);
  float g[VPL], sum[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) g[i] = sum[i] = 0.0f;
  R::store(s_row[wave], VPL * kWave, g);
  int seq = 0, seq_from = 0, seq_to = -1;  // none yet
  Tokens<VPL, VEC> tok;
  tok.weights = q.weights;
  tok.grad_weights = q.grad_weights;
  tok.init(q.logits, q.bias, q.ids, q.E, q.k, t0, t1, 1);
  while (tok.next()) {
    float* out = q.grad_logits + (size_t)tok.t * q.E;
    float d[VPL];
    const bool real = tok.real();
    if (__ballot(real) == 0) {  // a padded token, whatever its logits hold
#pragma unroll
      for (int i = 0; i < VPL; ++i) d[i] = 0.0f;
      R::template store<true>(out, q.E, d);
      continue;
    }
    if (q.counts && tok.t >= seq_to) {  // the first token, or past the sequence
      seq = seq_to < 0 ? 0 : seq + 1;
      if (seq < q.S && seq_end(q.seq_offsets, seq, q.T) <= tok.t)
        seq = sequence_at(q.seq_offsets, seq, q.S, tok.t);
      seq_from = seq < q.S ? seq_begin(q.seq_offsets, seq, q.T) : q.T;
      seq_to = seq < q.S ? seq_end(q.seq_offsets, seq, q.T) : q.T;
      if (seq < q.S) {
        int c[VPL];
        R::load(q.counts + (size_t)seq * q.E, q.E, c, 0);
        const float n = (float)max(q.tokens[seq], 1);
        const float f = (q.grad_loss ? q.grad_loss[0] : 1.0f) * (q.coef / (float)q.S) *
                        ((float)q.E / (float)q.k) / (n * n);
#pragma unroll
        for (int i = 0; i < VPL; ++i) g[i] = f * (float)c[i];
      }
    }
    float e[VPL], r[VPL], top;
    probabilities<VPL>(tok.l, q.score, e, r, top);
    const bool inside = q.counts && tok.t >= seq_from && seq < q.S;
    float total = 0.0f, weighted = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      total += e[i];
      weighted = fmaf(g[i], e[i], weighted);
    }
    const float w = real ? tok.w : 0.0f, gw = real ? tok.gw : 0.0f;
    total = wave_sum(total);
    weighted = wave_sum(weighted);
    const float inv = inside ? 1.0f / total : 0.0f;
    const float mean = weighted * inv;
#pragma unroll
    for (int i = 0; i < VPL; ++i) d[i] = e[i] * inv * (g[i] - mean);
    if (q.grad_weights) {
      // the slots' gradients change lanes through a row of zeros in LDS, which
      // is zero again afterwards (one wave's LDS accesses stay in order, and
      // those of one instruction to one address go by lane)
      const float dl = w * (gw - wave_sum(w * gw));
      if (real) atomicAdd(&s_row[wave][tok.id], dl);
      wave_lds_order();
      float add[VPL];
      R::load(s_row[wave], VPL * kWave, add, 0.0f);
      wave_lds_order();
      if (real) s_row[wave][tok.id] = 0.0f;
      wave_lds_order();
#pragma unroll
      for (int i = 0; i < VPL; ++i) d[i] += add[i];
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) d[i] *= r[i];
    R::template store<true>(out, q.E, d);
    if constexpr (BIAS) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum[i] += d[i];
    }
  }
  if constexpr (BIAS) {
    R::store(s_row[wave], VPL * kWave, sum);
    __syncthreads();
    float* part = static_cast<float*>(q.workspace) + (size_t)blockIdx.x * q.E;
    for (int e = threadIdx.x; e < q.E; e += kThreads)
      part[e] = s_row[0][e] + s_row[1][e] + s_row[2][e] + s_row[3][e];
  }
}

// 16 waves add up the blocks' sums of 64 experts.
__global__ void __launch_bounds__(kJoinWaves * kWave)
grad_bias_kernel(RouteGradParams q, int blocks) {
  __shared__ float s_sum[kJoinWaves][kWave];
  const int wave = threadIdx.x / kWave, lane = lane_id();
  const int e = blockIdx.x * kWave + lane;
  const float* parts = static_cast<const float*>(q.workspace);
  float sum = 0.0f;
  if (e < q.E) {
    const int per = (blocks + kJoinWaves - 1) / kJoinWaves;
    const int last = min((wave + 1) * per, blocks);
#pragma unroll 16
    for (int b = wave * per; b < last; ++b) sum += parts[(size_t)b * q.E + e];
  }
  s_sum[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || e >= q.E) return;
  float total = 0.0f;
  for (int i = 0; i < kJoinWaves; ++i) total += s_sum[i][lane];
  q.grad_bias[e] = total;
}

int grad_per_wave(int T) {
  const int waves = kGradBlocks * kWaves;
  return T <= waves ? 1 : (T + waves - 1) / waves;
}
int grad_blocks(int T) {
  const int per = grad_per_wave(T) * kWaves;
  return (T + per - 1) / per;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

// Values a lane: 1 up to 64 experts, then 4, 8 or 16, in 16-byte groups where
// rows and pointers are on 16-byte boundaries.
#define MOE_BY_WIDTH(E, ALIGNED, LAUNCH)       \
  do {                                         \
    if ((E) <= kWave) {                        \
      LAUNCH(1, 1);                            \
    } else if ((E) % 4 == 0 && (ALIGNED)) {    \
      if ((E) <= 4 * kWave) LAUNCH(4, 4);      \
      else if ((E) <= 8 * kWave) LAUNCH(8, 4); \
      else LAUNCH(16, 4);                      \
    } else {                                   \
      if ((E) <= 4 * kWave) LAUNCH(4, 1);      \
      else if ((E) <= 8 * kWave) LAUNCH(8, 1); \
      else LAUNCH(16, 1);                      \
    }                                          \
  } while (0)

size_t balance_workspace(int T, int E, int S) {
  if (one_block(T, S)) return 0;
  return parts_bytes(chunks_of(T), E, S);
}

hipError_t launch_balance_loss(const BalanceParams& q, hipStream_t st) {
  const bool aligned = aligned16(q.logits) && aligned16(q.bias);
  if (one_block(q.T, q.S)) {
#define MOE_LAUNCH(V, W)                                                                  \
  hipLaunchKernelGGL((balance_kernel<V, W, kOneBlockWaves, true>), dim3(1),               \
                     dim3(kOneBlockWaves * kWave), 0, st, q, Parts{}, q.T)
    MOE_BY_WIDTH(q.E, aligned, MOE_LAUNCH);
#undef MOE_LAUNCH
    return hipGetLastError();
  }
  const int chunk = chunk_tokens(q.T), chunks = chunks_of(q.T);
  const Parts parts = parts_of(q.workspace, chunks, q.E, q.S);
#define MOE_LAUNCH(V, W)                                                                      \
  hipLaunchKernelGGL((balance_kernel<V, W, kWaves, false>), dim3((unsigned)chunks),           \
                     dim3(kThreads), 0, st, q, parts, chunk)
  MOE_BY_WIDTH(q.E, aligned, MOE_LAUNCH);
#undef MOE_LAUNCH
  hipLaunchKernelGGL(balance_join_kernel,
                     dim3((unsigned)((q.E + kWave - 1) / kWave), (unsigned)(q.S < 4096 ? q.S : 4096)),
                     dim3(kJoinWaves * kWave), 0, st, q, parts, chunk);
  return hipGetLastError();
}

size_t route_grad_workspace(int T, int E) { return round16((size_t)grad_blocks(T) * E * 4); }

hipError_t launch_route_grad(const RouteGradParams& q, hipStream_t st) {
  const int blocks = grad_blocks(q.T), per_wave = grad_per_wave(q.T);
  const bool aligned = aligned16(q.logits) && aligned16(q.bias) && aligned16(q.grad_logits) &&
                       aligned16(q.counts);
  if (q.T > 0) {
#define MOE_LAUNCH(V, W)                                                                      \
  do {                                                                                        \
    if (q.grad_bias)                                                                          \
      hipLaunchKernelGGL((route_grad_kernel<V, W, true>), dim3((unsigned)blocks),             \
                         dim3(kThreads), 0, st, q, per_wave);                                 \
    else                                                                                      \
      hipLaunchKernelGGL((route_grad_kernel<V, W, false>), dim3((unsigned)blocks),            \
                         dim3(kThreads), 0, st, q, per_wave);                                 \
  } while (0)
    MOE_BY_WIDTH(q.E, aligned, MOE_LAUNCH);
#undef MOE_LAUNCH
  }
  if (q.grad_bias)
    hipLaunchKernelGGL(grad_bias_kernel, dim3((unsigned)((q.E + kWave - 1) / kWave)),
                       dim3(kJoinWaves * kWave), 0, st, q, blocks);
  return hipGetLastError();
}
#undef MOE_BY_WIDTH

}  // namespace moe
