// The gated linear recurrence (include/recur.h).
//
// A block takes a chunk of 64 positions (backward: 32) of 128 channels: 4 wavefronts of
// 16 (8) positions, a lane two channels.  A stretch of positions is h -> A h + H, so
// stretches join: positions in registers, wavefronts through LDS, chunks through words
// of the workspace that say by themselves when they are there (state_before).  Every
// input is read once and every output written once; the backward gets its states from
// one that the forward saved every 32 positions.
//
// Measured (bf16, 768 channels): forward of 131,072 positions 224 us (3.6 TB/s), of
// 49,152 86 us (3.5 TB/s); backward of 49,152 168 us (3.1 TB/s).  What bounds it is the
// time from a chunk's stretch to the state in front of it, two trips through memory
// that other blocks on the compute unit cover in part: without tickets and words the
// same kernels take 67 and 127 us, their vector instructions alone 43 and 85.  Hence
// few registers (three blocks a compute unit: 8 wavefronts of 8 positions each way, two
// and one block, took 117 and 228 us) and little to wait for.  A grid of resident blocks
// that load the next chunk ahead took 137 to 200 us forward: they drift apart, and one
// that is late holds tickets that all others wait for.
#include <algorithm>
#include <initializer_list>

#include "recur_dev.hpp"
#include "spans.hpp"

namespace recur {
namespace {

using spans::meet;
using spans::Span;

constexpr uint64_t kAlign = 256;

// Where sequences begin and end among the positions of a block's wavefronts: bit k is
// a wavefront's position k.
template <int WAVES, int STEPS>
struct Marks {
    uint32_t starts[WAVES], ends[WAVES];
    int start_of[WAVES][STEPS], end_of[WAVES][STEPS];   // the sequence, where the bit is set
};

// A wavefront's view of them, and which of its positions belong to a sequence.
struct Bits {
    uint32_t starts, ends, inside;
};

// Barrier that waits for LDS accesses only: a fence would wait for the rows' loads,
// which are on their way.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A sequence's first row and the one behind its last; read before the chunk's rows are
// asked for, because loads come back in order.
struct Ends {
    int32_t begin = 0, end = 0;

    __device__ __forceinline__ void load(const Args &a, int64_t s)
    {
        begin = end = 0;
        if (a.offsets && s < a.n) {
            begin = a.offsets[s];
            end = a.offsets[s + 1];
        }
    }
};

// All threads of the block; mine: the sequence of the thread's own number.  The
// sequences that can matter, where there are many: those from the last probe that
// begins in front of t0 to the first that begins behind the chunk.
template <int WAVES, int STEPS>
__device__ __forceinline__ void find_marks(const Args &a, int64_t t0, Ends mine, Marks<WAVES, STEPS> *m)
{
    constexpr int threads = WAVES * 64, N = WAVES * STEPS;
    __shared__ int from, to;
    if (threadIdx.x < WAVES)
        m->starts[threadIdx.x] = m->ends[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
        from = 0;
        to = (int)a.n;
    }
    lds_barrier();
    auto mark = [&](int s, const Ends &k) {
        const int64_t b = (int64_t)k.begin - t0, e = (int64_t)k.end - t0 - 1;   // first and last position
        if (b > e)
            return;
        if (b >= 0 && b < N) {
            atomicOr(&m->starts[b / STEPS], 1u << (b % STEPS));
            m->start_of[b / STEPS][b % STEPS] = s;
        }
        if (e >= 0 && e < N) {
            atomicOr(&m->ends[e / STEPS], 1u << (e % STEPS));
            m->end_of[e / STEPS][e % STEPS] = s;
        }
    };
    if (a.n <= 4 * threads) {
        mark((int)threadIdx.x, mine);
        for (int s = threads + (int)threadIdx.x; s < a.n; s += threads) {
            mine.load(a, s);
            mark(s, mine);
        }
    } else {
        const int64_t step = (a.n + threads - 1) / threads, at = threadIdx.x * step;
        if (at < a.n) {
            const int32_t v = a.offsets[at];
            if (v < t0)
                atomicMax(&from, (int)at);
            if (v > t0 + N)
                atomicMin(&to, (int)at);
        }
        lds_barrier();
        for (int s = from + (int)threadIdx.x; s < to; s += threads) {
            mine.load(a, s);
            mark(s, mine);
        }
    }
    lds_barrier();
}

// The block's chunk, and its column of channels.  A block that waits for others takes
// its chunk when it begins to run, in the order in which a column's chunks depend on one
// another: whoever it waits for has begun before it.  A ticket a column, each in a line of
// its own: one address gives out a number every 18 ns, which with one ticket for all
// bounded the kernels (backward of 4,096 x 768 28.1 us instead of 21.2, forward of 16,384
// 42.9 instead of 34.4).
__device__ __forceinline__ void place(const Args &a, int &chunk, int &column)
{
    __shared__ uint32_t ticket;
    chunk = 0;
    column = blockIdx.x;
    if (!a.alone) {
        column = blockIdx.x % (uint32_t)a.columns;
        if (threadIdx.x == 0)
            ticket = atomicAdd(a.tickets + column * kTicketWords, 1u);
        __syncthreads();
        chunk = (int)ticket;
    }
}

// The rows that belong to a sequence.
__device__ __forceinline__ void rows_of_sequences(const Args &a, int64_t &lo, int64_t &hi)
{
    lo = a.offsets ? max((int64_t)0, (int64_t)a.offsets[0]) : 0;
    hi = a.offsets ? max((int64_t)0, min(a.T, (int64_t)a.offsets[a.n])) : a.T;
}

// t: the wavefront's first position.
template <int WAVES, int STEPS>
__device__ __forceinline__ Bits bits_of(const Args &a, const Marks<WAVES, STEPS> &m, int64_t t, int64_t lo, int64_t hi,
                                        int wave)
{
    Bits b;
    if (a.offsets) {
        b.starts = m.starts[wave];
        b.ends = m.ends[wave];
    } else {
        b.starts = t == 0 ? 1u : 0u;
        b.ends = hi > t && hi <= t + STEPS ? 1u << (hi - 1 - t) : 0u;
    }
    b.inside = (1u << STEPS) - 1;
    if (t < lo || t + STEPS > hi) {
        b.inside = 0;
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
            b.inside |= (t + k >= lo && t + k < hi ? 1u : 0u) << k;
    }
    b.starts = __builtin_amdgcn_readfirstlane(b.starts & b.inside);
    b.ends = __builtin_amdgcn_readfirstlane(b.ends & b.inside);
    b.inside = __builtin_amdgcn_readfirstlane(b.inside);
    return b;
}

template <int V, int WAVES, int STEPS>
struct Shared {
    Span1 waves[WAVES][V][64];    // each wavefront's stretch
    Span1 before[WAVES][V][64];   // stretches of the chunks before, some to a wavefront
    Span1 all[V][64];             // the chunk
    float state[V][64];           // the state in front of the group of chunks
    Marks<WAVES, STEPS> marks;
};

// The state in front of the block's chunk; `index` counts chunks in the order in
// which they depend on one another.  own: the wavefront's stretch, `order` its
// place in the block in that order.
//
// Every chunk says what it does to a state (sums) as soon as it knows it, without
// waiting for anyone; the last chunk of a group of kGroup says what state it leaves
// (states), so only those form a chain, and one of them hands on as soon as the one
// before has.  A chunk takes the state in front of its group through the group's
// earlier chunks, always in the same order: results do not depend on who came
// first.  (Groups of 32 and 64: 175 and 210 us instead of 171 for the backward of
// 49,152 positions, 21.9 and 28.0 instead of 21.3 for 4,096.)  A wait ends: who is
// waited for has begun to run (place), and waits itself only for chunks in front of it;
// should one never answer, the values become NaN after a bounded number of polls.
constexpr int kPolls = 1 << 20;

__device__ __forceinline__ uint64_t wait_for(const uint64_t *p, uint64_t w)
{
    for (int polls = 0; polls < kPolls && __any(w == kNone); ++polls) {
        __builtin_amdgcn_s_sleep(1);
        if (w == kNone)
            w = peek(p);
    }
    return w;
}

template <int V, int WAVES, int STEPS>
__device__ __forceinline__ void state_before(const Args &a, Shared<V, WAVES, STEPS> &sh, int index, int column,
                                             int wave, int order, int lane, const Span1 (&own)[V], float (&h)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v)
        sh.waves[order][v][lane] = own[v];
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v)
        h[v] = 0.0f;
    if (a.alone)
        return;
    constexpr int per = (kGroup + WAVES - 1) / WAVES;
    const int group = index / kGroup, place = index % kGroup;
    const int64_t step = (int64_t)a.columns * V * 64;   // words of a chunk
    const int at = column * V * 64 + lane;
    if (wave == WAVES - 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            Span1 all = sh.waves[0][v][lane];
#pragma unroll
            for (int w = 1; w < WAVES; ++w)
                all = join(all, sh.waves[w][v][lane]);
            publish(&a.sums[index * step + at + v * 64], word(all));
            sh.all[v][lane] = all;
        }
    }
    if (place > 0) {
        const uint64_t *p = a.sums + ((int64_t)group * kGroup + wave * per) * step + at;
        const int mine = min(per, place - wave * per);   // chunks before that this wavefront looks at
        const bool asks = wave == WAVES - 1 && group > 0;
        const uint64_t *q = a.states + group * step + at;
        uint64_t first[V];
        uint64_t w[per][V];
#pragma unroll
        for (int i = 0; i < per; ++i)
            if (i < mine)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    w[i][v] = peek(p + i * step + v * 64);
        if (asks)   // mostly there by now
#pragma unroll
            for (int v = 0; v < V; ++v)
                first[v] = peek(q + v * 64);
        Span1 s[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
            s[v] = Span1{1.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < per; ++i)
            if (i < mine)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    s[v] = join(s[v], span(wait_for(p + i * step + v * 64, w[i][v])));
#pragma unroll
        for (int v = 0; v < V; ++v)
            sh.before[wave][v][lane] = s[v];
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v)
            s[v] = sh.before[0][v][lane];
        for (int i = 1; i * per < place; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v)
                s[v] = join(s[v], sh.before[i][v][lane]);
        // where a sequence began in between (the same for all channels), nothing in front counts
        const bool cut = __all(s[0].A < 0.0f);
        if (wave == WAVES - 1) {
            if (asks && !cut)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    h[v] = span(wait_for(q + v * 64, first[v])).H;
            if (place == kGroup - 1 && index + 1 < a.chunks)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    publish(a.states + (group + 1) * step + at + v * 64,
                            word(Span1{1.0f, through(sh.all[v][lane], through(s[v], h[v]))}));
        }
        if (group > 0 && !cut) {
            if (wave == WAVES - 1)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    sh.state[v][lane] = h[v];
            __syncthreads();
#pragma unroll
            for (int v = 0; v < V; ++v)
                h[v] = sh.state[v][lane];
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            h[v] = through(s[v], h[v]);
    } else if (group > 0) {
        if (wave == WAVES - 1) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                sh.state[v][lane] = span(wait_for(a.states + group * step + at + v * 64, kNone)).H;
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v)
            h[v] = sh.state[v][lane];
    }
}

// Clears the words that blocks wait for, and gives sequences without rows their
// states: out = in (or 0).
__global__ __launch_bounds__(256) void clear_kernel(Args a, const float *in, float *out)
{
    const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    if (!a.alone) {
        ulonglong2 *sums = reinterpret_cast<ulonglong2 *>(a.sums);   // sums, then states: a multiple of 64 words
        for (int64_t k = first; k < a.words / 2; k += step)
            sums[k] = make_ulonglong2(kNone, kNone);
        for (int64_t k = first; k < a.columns; k += step)
            a.tickets[k * kTicketWords] = 0;
    }
    if (out) {
        for (int64_t s = blockIdx.x; s < a.n; s += gridDim.x) {
            const int64_t b = a.offsets ? a.offsets[s] : 0, e = a.offsets ? a.offsets[s + 1] : a.T;
            if (b < e)
                continue;
            for (int j = threadIdx.x; j < a.D; j += 256)
                out[s * a.D + j] = in ? in[s * a.D + j] : 0.0f;
        }
    }
}

// STEPS rows from t on; rows behind the last are the last again.
template <int E, int V, int STEPS>
__device__ __forceinline__ void load_rows(const uint8_t *p, int64_t ld, int64_t t, int64_t T, uint32_t off,
                                          Raw<E, V> (&v)[STEPS])
{
    p += t * ld;
    if (t + STEPS <= T) {
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            v[k] = load<E, V>(p + off);
            p += ld;
        }
    } else {
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
            v[k] = load<E, V>(p + (min(t + k, T - 1) - t) * ld + off);
    }
}

// all: every z of the wavefront, at all of its positions, is above kSeries.
template <int E, int V>
__device__ __forceinline__ void fwd_gates(const Raw<E, V> (&x)[kFwdSteps], const Raw<E, V> (&r)[kFwdSteps],
                                          const Raw<E, V> (&i)[kFwdSteps], const float (&rate)[V], bool all,
                                          float (&av)[kFwdSteps][V], float (&u)[kFwdSteps][V])
{
#pragma unroll
    for (int k = 0; k < kFwdSteps; ++k) {
        float xf[V], rf[V], gf[V], z[V], e[V];
        unpack<E, V>(x[k], xf);
        unpack<E, V>(r[k], rf);
        unpack<E, V>(i[k], gf);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            z[v] = rate[v] * sigmoid(rf[v]);
            decay_near(z[v], av[k][v], e[v]);
        }
        if (!all) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                decay_any(z[v], av[k][v], e[v]);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            u[k][v] = rest_of(e[v]) * sigmoid(gf[v]) * xf[v];
            here(av[k][v]);
            here(u[k][v]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Rows are asked for before anything else is looked at, and stay packed until their gates
// are computed; a_t and u_t of all positions then stay in registers until the state in
// front is known.  One exp for each gate and one more beyond kSeries, one square root.
template <int E, int V, int WAVES>
__global__ __launch_bounds__(WAVES * 64, E == 2 && WAVES == kWaves ? 3 : 2) void fwd_kernel(Args a)
{
    constexpr int STEPS = kFwdSteps, N = WAVES * STEPS;
    __shared__ Shared<V, WAVES, STEPS> sh;
    int chunk, column;
    place(a, chunk, column);
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    // lanes past the last channels take those again: the same loads, values and stores
    const int j = min((column * 64 + lane) * V, a.D - V);
    const uint32_t off = (uint32_t)j * E;   // behind a row's address, which is the same for all lanes
    const int64_t t0 = (int64_t)chunk * N, t = t0 + wave * STEPS;
    Ends mine;
    mine.load(a, threadIdx.x);
    __builtin_amdgcn_sched_barrier(0);
    Raw<E, V> x[STEPS], r[STEPS], i[STEPS];
    load_rows<E, V, STEPS>(a.r, a.ldr, t, a.T, off, r);
    load_rows<E, V, STEPS>(a.i, a.ldi, t, a.T, off, i);
    load_rows<E, V, STEPS>(a.x, a.ldx, t, a.T, off, x);
    float rate[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        rate[v] = decay(a.lam[j + v], a.c);
    int64_t lo, hi;
    rows_of_sequences(a, lo, hi);
    if (t0 >= hi)
        return;   // nor does any chunk behind it ask
    if (a.offsets)
        find_marks<WAVES, STEPS>(a, t0, mine, &sh.marks);
    const Bits bits = bits_of<WAVES, STEPS>(a, sh.marks, t, lo, hi, wave);
    const bool plain = bits.starts == 0 && bits.ends == 0 && bits.inside == (1u << STEPS) - 1;
    float av[STEPS][V], u[STEPS][V];
    bool all = true;
#pragma unroll
    for (int v = 0; v < V; ++v)
        all = all && rate[v] > kSeries;
    // One channel a lane: a copy of the loop for slow decays and one for any (1,000 x 770
    // bf16: 8.8 us instead of 9.1).  Two: a branch a position in one loop, because the results
    // of two copies cannot take the packed rows' registers (172 instead of 137 with fp32,
    // 136 us instead of 128 for 49,152 x 768; bf16 with a channel of fast decay 94 instead of
    // 90, 16,384 x 768 without one 34.3 instead of 34.7).
    const bool slow = __all(all);
    if constexpr (V == 1) {
        if (slow)
            fwd_gates<E, V>(x, r, i, rate, true, av, u);
        else
            fwd_gates<E, V>(x, r, i, rate, false, av, u);
    } else {
        fwd_gates<E, V>(x, r, i, rate, slow, av, u);
    }
    Span1 own[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        own[v] = Span1{1.0f, 0.0f};
    if (plain) {
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                own[v].A *= av[k][v];
                own[v].H = __builtin_fmaf(av[k][v], own[v].H, u[k][v]);
            }
    } else {
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const bool start = bits.starts >> k & 1, inside = bits.inside >> k & 1;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                av[k][v] = inside ? av[k][v] : 1.0f;
                u[k][v] = inside ? u[k][v] : 0.0f;
            }
            if (start && a.h0) {
                const int64_t s = a.offsets ? sh.marks.start_of[wave][k] : 0;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    u[k][v] = __builtin_fmaf(av[k][v], a.h0[s * a.D + j + v], u[k][v]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                own[v].A *= av[k][v];
                own[v].H = start ? u[k][v] : __builtin_fmaf(av[k][v], own[v].H, u[k][v]);
            }
        }
        if (bits.starts) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                own[v].A = -1.0f;
        }
    }
    float h[V];
    state_before<V, WAVES, STEPS>(a, sh, chunk, column, wave, wave, lane, own, h);
    for (int w = 0; w < wave; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v)
            h[v] = through(sh.waves[w][v][lane], h[v]);
    // the wavefront's position in front of which a state is saved, if one is: RECUR_CHUNK >= STEPS
    const int keep = a.saved ? (int)((RECUR_CHUNK - t % RECUR_CHUNK) % RECUR_CHUNK) : STEPS;
    float *saved = a.saved + (t + keep) / RECUR_CHUNK * a.D + j;
    auto save = [&](int k) {
        if (k == keep && t + k < a.T) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                saved[v] = h[v];
        }
    };
    uint8_t *y = a.y + t * a.D * E;
    if (plain) {
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            save(k);
#pragma unroll
            for (int v = 0; v < V; ++v)
                h[v] = __builtin_fmaf(av[k][v], h[v], u[k][v]);
            store<E, V>(y + off, h);
            y += (int64_t)a.D * E;
        }
    } else {
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            save(k);
#pragma unroll
            for (int v = 0; v < V; ++v)
                h[v] = bits.starts >> k & 1 ? u[k][v] : __builtin_fmaf(av[k][v], h[v], u[k][v]);
            if (bits.inside >> k & 1)
                store<E, V>(y + off, h);
            y += (int64_t)a.D * E;
            if (a.hT && (bits.ends >> k & 1)) {
                const int64_t s = a.offsets ? sh.marks.end_of[wave][k] : 0;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    a.hT[s * a.D + j + v] = h[v];
            }
        }
    }
}

// The sequence that begins or ends at the wavefront's position k.
__device__ __forceinline__ int64_t sequence_of(const Args &a, const int *of, int k) { return a.offsets ? of[k] : 0; }

// H = the sequence's row of h0 or dhT, 0 without them.
template <int V>
__device__ __forceinline__ void row_of(const float *p, int64_t sequence, int D, int j, Span1 (&to)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v)
        to[v].H = p ? p[sequence * D + j + v] : 0.0f;
}

// A channel's dlam from its sum of rho dz.
__device__ __forceinline__ void put_dlam(const Args &a, int j, float sum)
{
    const float v = alone(-a.c * sigmoid(a.lam[j]), sum);
    a.dlam[j] = a.accum ? a.dlam[j] + v : v;
}

// A position's numbers that need no state: a, m g (dx / G), m g x (1 - g) (di / G), and
// of dz / G the part beside a h_{t-1}: g x a^2 / m.
template <int E, int V, bool ALL>
__device__ __forceinline__ void bwd_gates(const Raw<E, V> (&x)[kBwdSteps], const Raw<E, V> (&r)[kBwdSteps],
                                          const Raw<E, V> (&i)[kBwdSteps], const float (&rate)[V], float (&av)[kBwdSteps][V],
                                          float (&c1)[kBwdSteps][V], float (&c2)[kBwdSteps][V],
                                          float (&c3)[kBwdSteps][V], float (&cr)[kBwdSteps][V], float (&cl)[kBwdSteps][V])
{
#pragma unroll
    for (int k = 0; k < kBwdSteps; ++k) {
        float xf[V], rf[V], gf[V];
        unpack<E, V>(x[k], xf);
        unpack<E, V>(r[k], rf);
        unpack<E, V>(i[k], gf);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float rho, rho_rest, g, g_rest, m;
            sigmoid(rf[v], rho, rho_rest);
            sigmoid(gf[v], g, g_rest);
            const float z = rate[v] * rho;
            decays<ALL>(z, av[k][v], m);
            c1[k][v] = m * g;
            c2[k][v] = c1[k][v] * xf[v] * g_rest;
            cl[k][v] = rho;
            cr[k][v] = z * rho_rest;
            // 0 where m is (z is too): a large number instead would make an infinity of a large x
            const float over = m > 0.0f ? __builtin_amdgcn_rcpf(m) : 0.0f;
            c3[k][v] = g * xf[v] * (av[k][v] * av[k][v] * over);
            here(av[k][v]);
            here(c1[k][v]);
            here(c2[k][v]);
            here(c3[k][v]);
            here(cl[k][v]);
            here(cr[k][v]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Chunks from the last to the first.  The states come from the saved one, forward
// through the chunk; with them and the gates every output is G_t times a number of
// its position: dx c1, di c2, dr cr, and rho dz (of dlam) cl.  G in turn runs
// backwards, what a position hands on being a_t G_t.  Those four numbers are all that
// the registers keep over the wait (168 of them with bf16).  One channel a lane and 16
// positions instead: 358 us of 49,152 x 768 instead of 176 (spills, and half the bytes a
// load).
template <int E, int V, int WAVES>
__global__ __launch_bounds__(WAVES * 64, WAVES == kWaves ? 3 : 2) void bwd_kernel(Args a)
{
    constexpr int STEPS = kBwdSteps, N = WAVES * STEPS;
    __shared__ Shared<V, WAVES, STEPS> sh;
    int index, column;
    place(a, index, column);
    int64_t lo, hi;
    rows_of_sequences(a, lo, hi);
    const int chunk = a.chunks - 1 - index;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int j = min((column * 64 + lane) * V, a.D - V);
    const uint32_t off = (uint32_t)j * E;
    const int64_t t0 = (int64_t)chunk * N, t = t0 + wave * STEPS;
    Ends mine;
    mine.load(a, threadIdx.x);
    __builtin_amdgcn_sched_barrier(0);
    Raw<E, V> x[STEPS], r[STEPS], i[STEPS], d[STEPS];
    load_rows<E, V, STEPS>(a.r, a.ldr, t, a.T, off, r);
    load_rows<E, V, STEPS>(a.i, a.ldi, t, a.T, off, i);
    load_rows<E, V, STEPS>(a.x, a.ldx, t, a.T, off, x);
    load_rows<E, V, STEPS>(a.dy, (int64_t)a.D * E, t, a.T, off, d);
    float rate[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        rate[v] = decay(a.lam[j + v], a.c);
        h[v] = a.saved[(int64_t)chunk * a.D + j + v];
    }
    if (a.offsets)
        find_marks<WAVES, STEPS>(a, t0, mine, &sh.marks);
    const Bits bits = bits_of<WAVES, STEPS>(a, sh.marks, t, lo, hi, wave);
    const bool plain = bits.starts == 0 && bits.ends == 0 && bits.inside == (1u << STEPS) - 1;
    float av[STEPS][V], c1[STEPS][V], c2[STEPS][V], c3[STEPS][V], cr[STEPS][V], cl[STEPS][V];
    bool all = true;
#pragma unroll
    for (int v = 0; v < V; ++v)
        all = all && rate[v] > kSeries;
    if (__all(all))
        bwd_gates<E, V, true>(x, r, i, rate, av, c1, c2, c3, cr, cl);
    else
        bwd_gates<E, V, false>(x, r, i, rate, av, c1, c2, c3, cr, cl);
    // forward: what the stretch does to a state; backward: what reaches it from behind
    // goes to A in + H, with the same A
    Span1 own[V], back[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        own[v] = Span1{1.0f, 0.0f};
        back[v].H = 0.0f;
    }
    if (plain) {
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            float xf[V];
            unpack<E, V>(x[k], xf);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                own[v].A *= av[k][v];
                own[v].H = __builtin_fmaf(av[k][v], own[v].H, c1[k][v] * xf[v]);
            }
        }
#pragma unroll
        for (int k = STEPS - 1; k >= 0; --k) {
            float df[V];
            unpack<E, V>(d[k], df);
#pragma unroll
            for (int v = 0; v < V; ++v)
                back[v].H = av[k][v] * (df[v] + back[v].H);
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            back[v].A = own[v].A;
    } else {
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            if (!(bits.inside >> k & 1)) {
                x[k].w = d[k].w = 0;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    av[k][v] = 1.0f;
            }
            if (bits.starts >> k & 1)
                row_of<V>(a.h0, sequence_of(a, sh.marks.start_of[wave], k), a.D, j, own);
            float xf[V];
            unpack<E, V>(x[k], xf);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                own[v].A *= av[k][v];
                own[v].H = __builtin_fmaf(av[k][v], own[v].H, c1[k][v] * xf[v]);
            }
        }
#pragma unroll
        for (int k = STEPS - 1; k >= 0; --k) {
            if (bits.ends >> k & 1)
                row_of<V>(a.dhT, sequence_of(a, sh.marks.end_of[wave], k), a.D, j, back);
            float df[V];
            unpack<E, V>(d[k], df);
#pragma unroll
            for (int v = 0; v < V; ++v)
                back[v].H = av[k][v] * (df[v] + back[v].H);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            back[v].A = bits.ends ? -1.0f : own[v].A;
            own[v].A = bits.starts ? -1.0f : own[v].A;
        }
    }
    // h_{t-1}, and what it makes of the numbers above
#pragma unroll
    for (int v = 0; v < V; ++v)
        sh.before[wave][v][lane] = own[v];
    __syncthreads();
    for (int w = 0; w < wave; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v)
            h[v] = through(sh.before[w][v][lane], h[v]);
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        if (bits.starts >> k & 1) {
            row_of<V>(a.h0, sequence_of(a, sh.marks.start_of[wave], k), a.D, j, own);
#pragma unroll
            for (int v = 0; v < V; ++v)
                h[v] = own[v].H;
        }
        float xf[V];
        unpack<E, V>(x[k], xf);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float ah = av[k][v] * h[v], z = ah - c3[k][v];   // z: dz / G
            cr[k][v] *= z;
            cl[k][v] *= z;
            here(cr[k][v]);
            here(cl[k][v]);
            h[v] = __builtin_fmaf(c1[k][v], xf[v], ah);
        }
    }
    float in[V], acc[V];
    state_before<V, WAVES, STEPS>(a, sh, index, column, wave, WAVES - 1 - wave, lane, back, in);
    for (int w = 0; w < WAVES - 1 - wave; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v)
            in[v] = through(sh.waves[w][v][lane], in[v]);
#pragma unroll
    for (int v = 0; v < V; ++v)
        acc[v] = 0.0f;
    uint8_t *px = a.dx + (t + STEPS - 1) * a.lddx, *pr = a.dr + (t + STEPS - 1) * a.lddr,
            *pi = a.di + (t + STEPS - 1) * a.lddi;
#pragma unroll
    for (int k = STEPS - 1; k >= 0; --k) {
        if (bits.ends >> k & 1) {
            row_of<V>(a.dhT, sequence_of(a, sh.marks.end_of[wave], k), a.D, j, own);
#pragma unroll
            for (int v = 0; v < V; ++v)
                in[v] = own[v].H;
        }
        float df[V], dx[V], di[V], dr[V], dl[V];
        unpack<E, V>(d[k], df);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float G = df[v] + in[v];
            in[v] = av[k][v] * G;
            dx[v] = G * c1[k][v];
            di[v] = G * c2[k][v];
            dr[v] = G * cr[k][v];
            dl[v] = G * cl[k][v];
        }
        if (bits.inside >> k & 1) {
            store<E, V>(px + off, dx);
            store<E, V>(pi + off, di);
            store<E, V>(pr + off, dr);
#pragma unroll
            for (int v = 0; v < V; ++v)
                acc[v] += dl[v];
        }
        px -= a.lddx;
        pr -= a.lddr;
        pi -= a.lddi;
        if (a.dh0 && (bits.starts >> k & 1)) {
            const int64_t s = a.offsets ? sh.marks.start_of[wave][k] : 0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                a.dh0[s * a.D + j + v] = in[v];
        }
    }
    __syncthreads();   // every wavefront has gone through sh.waves
#pragma unroll
    for (int v = 0; v < V; ++v)
        sh.waves[wave][v][lane].A = acc[v];
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float s = sh.waves[0][v][lane].A;
#pragma unroll
            for (int w = 1; w < WAVES; ++w)
                s += sh.waves[w][v][lane].A;
            if (V == 1 && a.alone) {   // the only chunk: one channel a lane
                if (column * 64 + lane < a.D)   // it may add to what is there: once
                    put_dlam(a, j, s);
            } else {
                a.part[(int64_t)chunk * a.D + j + v] = s;
            }
        }
    }
}

// dlam from the chunks' parts, in a fixed order: 16 channels a block, 64 threads to
// a channel.
__global__ __launch_bounds__(1024) void dlam_kernel(Args a)
{
    __shared__ float lds[16][16];
    const int c = threadIdx.x % 16, g = threadIdx.x / 16, j = blockIdx.x * 16 + c;
    float s = 0.0f;
    if (j < a.D) {
#pragma unroll 16
        for (int64_t k = g; k < a.chunks; k += 64)
            s += a.part[k * a.D + j];
    }
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (g % 4 == 0)
        lds[g / 4][c] = s;
    __syncthreads();
    if (g != 0 || j >= a.D)
        return;
#pragma unroll
    for (int k = 1; k < 16; ++k)
        s += lds[k][c];
    put_dlam(a, j, s);
}

// The rows of one slot: whether `row` is the first of them (it takes them all, in
// order), and `more`: whether others follow.  Eight loads of 64 slots at a time, the last
// slot again behind the end: as many for every lane, or the rest would be loaded one by
// one (500 rows of 2,048 channels: 8.9 us instead of 6.6; without looking 5.5).  Every
// wavefront looks at all n slots, so many rows cost n^2: calls of 768 channels take 9.4 us
// for 1,024 rows, 13.5 for 2,048, 33 for 4,096, 340 for 16,384 and 5,030 for 65,536,
// without slots 8.6, 8.2, 11, 33 and 149.
__device__ __forceinline__ bool first_of_slot(const int32_t *slots, int n, int row, int slot, int lane, bool &more)
{
    bool before = false, behind = false;
    for (int at = 0; at < n; at += 512) {
        int32_t s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s[i] = slots[min(at + i * 64 + lane, n - 1)];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = min(at + i * 64 + lane, n - 1);
            before = before || (s[i] == slot && k < row);
            behind = behind || (s[i] == slot && k > row);
        }
    }
    more = __any(behind);
    return !__any(before);
}

// The next row of the slot behind `row`, n if there is none.  (Slot by slot instead: 44 us
// instead of 9.3 for 500 rows of which each two share a slot, 600 instead of 44 for 4,096.)
__device__ __forceinline__ int next_of_slot(const int32_t *slots, int n, int row, int slot, int lane)
{
    for (int at = row + 1; at < n; at += 512) {
        int32_t s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s[i] = slots[min(at + i * 64 + lane, n - 1)];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t hit = __ballot(s[i] == slot && at + i * 64 + lane < n);
            if (hit)
                return at + i * 64 + __builtin_ctzll(hit);
        }
    }
    return n;
}

// A wavefront takes a row and V channels a lane; D is a multiple of V: the state is read
// and written in place, so no channel may be two wavefronts'.
template <int E, int V>
__global__ __launch_bounds__(256) void step_kernel(Args a, float *state, int states, const int32_t *slots, int n)
{
    const int unit = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int row = unit / a.columns;
    if (row >= n)
        return;
    const int mine = (unit % a.columns * 64 + lane) * V, j = min(mine, a.D - V);
    const uint32_t off = (uint32_t)j * E;
    Raw<E, V> x = load<E, V>(a.x + row * a.ldx + off), r = load<E, V>(a.r + row * a.ldr + off),
              i = load<E, V>(a.i + row * a.ldi + off);
    float rate[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        rate[v] = decay(a.lam[j + v], a.c);
    const int slot = slots ? __builtin_amdgcn_readfirstlane(slots[row]) : row;
    const int64_t y = (int64_t)a.D * E;
    if (slot < 0 || slot >= states) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            h[v] = 0.0f;
        store<E, V>(a.y + row * y + off, h);
        return;
    }
    float *s = state + (int64_t)slot * a.D;
#pragma unroll
    for (int v = 0; v < V; ++v)
        h[v] = s[(uint32_t)(j + v)];
    bool more = false;
    if (slots && !first_of_slot(slots, n, row, slot, lane, more))
        return;
    for (int t = row;;) {
        float xf[V], rf[V], gf[V];
        unpack<E, V>(x, xf);
        unpack<E, V>(r, rf);
        unpack<E, V>(i, gf);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float d, m;
            decays<false>(rate[v] * sigmoid(rf[v]), d, m);
            h[v] = __builtin_fmaf(d, h[v], m * sigmoid(gf[v]) * xf[v]);
        }
        store<E, V>(a.y + t * y + off, h);
        if (!more)
            break;
        t = next_of_slot(slots, n, t, slot, lane);
        if (t >= n)
            break;
        x = load<E, V>(a.x + t * a.ldx + off);
        r = load<E, V>(a.r + t * a.ldr + off);
        i = load<E, V>(a.i + t * a.ldi + off);
    }
    if (mine < a.D) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            s[(uint32_t)(j + v)] = h[v];
    }
}

uint64_t size_of(int dtype) { return dtype == RECUR_DTYPE_F32 ? 4 : 2; }

int check_config(const recur_config *c)
{
    if (!c)
        return RECUR_ENULL;
    const bool ok = c->dim >= 1 && c->dim <= 16384 && (c->dtype == RECUR_DTYPE_F32 || c->dtype == RECUR_DTYPE_BF16) &&
                    c->c > 0.0f && c->c <= 64.0f && (c->options & ~RECUR_OPT_ACCUM) == 0 && c->max_tokens >= 1 &&
                    c->max_tokens <= (int64_t(1) << 24);
    return ok ? RECUR_OK : RECUR_ECONFIG;
}

int64_t saved_rows(int64_t T) { return (T + RECUR_CHUNK - 1) / RECUR_CHUNK; }
// Wavefronts of a block: the usual ones, or many where a call that they have not room
// for is then one chunk, with no words to clear and nobody to wait for (calls back to
// back, 768 channels: forward of 100 positions 11.6 us instead of 14.6, of 250 11.5 instead
// of 14.3, forward and backward of 100 26.4 instead of 35.1; without the results' allocation,
// 64 to 8,192 channels alike: forward of 250 8.5 to 9.2 instead of 11.0 to 11.4, backward of
// 40 and 120 11.5 to 12.1 instead of 18.1 to 18.4).
int waves(int pass, int64_t T)
{
    const int steps = pass == RECUR_PASS_FWD ? kFwdSteps : kBwdSteps;
    return T > kWaves * steps && T <= kManyWaves * steps ? kManyWaves : kWaves;
}
int64_t chunk_of(int pass, int64_t T) { return waves(pass, T) * (pass == RECUR_PASS_FWD ? kFwdSteps : kBwdSteps); }
int64_t chunks(int pass, int64_t T) { return (T + chunk_of(pass, T) - 1) / chunk_of(pass, T); }
uint64_t align_up(uint64_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

// Channels of a lane: two, but one up to 64 channels, where half the wavefront would
// have none, and for as few blocks (or rows of a step) that twice as many still run at once
// (backward of 2,048 x 768 bf16, 384 blocks: 13.8 us instead of 16.0; of 3,000, 564: 20.2
// instead of 19.8; forward of 4,096, 384: 12.8 instead of 15.1; of 6,000, 564: 19.6 instead
// of 18.7; backward of 49,152: 196 instead of 171).  At 256, 2,048 and 8,192 channels one is
// within 2 % of two or faster up to 400 blocks as well (calls of 12,800 x 256 17.9 instead of
// 23.1, 1,600 x 2,048 12.5 instead of 13.9, 384 x 8,192 11.3 instead of 12.4), and of 256 channels
// further on (28,800 forward 31.6 instead of 41.3): there the limit gives time away.
constexpr int64_t kFewBlocks = 400;
int per_lane(int D, int64_t rows) { return D <= 64 || rows * ((D + 127) / 128) <= kFewBlocks ? 1 : 2; }
// Of a pass: one too where the call is one chunk, whose 1,024 threads have 128 registers,
// and in the backward of fp32, where two take 190, two blocks a compute unit instead of
// four (4,096 x 768: 25.3 us instead of 29.0, 16,384: 84.9 instead of 88.7, 49,152: 252
// instead of 254; the forward's 137 leave it three, and of 49,152 it takes 128 instead of 139).
int per_lane(const recur_config *c, int pass, int64_t n)
{
    return n <= 1 || (pass == RECUR_PASS_BWD && c->dtype == RECUR_DTYPE_F32) ? 1 : per_lane(c->dim, n);
}
int64_t columns(int D, int per) { return (D + 64 * per - 1) / (64 * per); }

// Workspace: the tickets, the words of n chunks and their groups, the backward's
// parts of dlam.  Words of a row of chunks: enough for one or two channels a lane.
uint64_t row_words(int D) { return (uint64_t)columns(D, 2) * 128; }
uint64_t words_of(int D, int64_t n) { return (uint64_t)(n + n / kGroup + 1) * row_words(D); }
// One or two channels a lane: no more columns than 64 channels each make.
uint64_t ticket_bytes(int D) { return align_up((uint64_t)columns(D, 1) * kTicketWords * 4); }
uint64_t ws_need(const recur_config *c, int pass)
{
    const int64_t n = chunks(pass, c->max_tokens);
    return ticket_bytes(c->dim) + align_up(words_of(c->dim, n) * 8) +
           (pass == RECUR_PASS_BWD ? align_up((uint64_t)n * c->dim * 4) : 0);
}

struct Buf {
    Span s;
    uint64_t elt;
    bool needed;
};

int check(std::initializer_list<Buf> ins, std::initializer_list<Buf> outs, const Span &ws)
{
    for (const auto *l : {&ins, &outs})
        for (const Buf &b : *l) {
            if (b.needed && !b.s.p && b.s.len && b.s.rows)
                return RECUR_ENULL;
            if ((uintptr_t)b.s.p % b.elt)
                return RECUR_EALIGN;
        }
    const Buf *o = outs.begin();
    for (size_t i = 0; i < outs.size(); ++i) {
        for (const Buf &b : ins)
            if (meet(o[i].s, b.s))
                return RECUR_EARG;
        for (size_t k = 0; k < i; ++k)
            if (meet(o[i].s, o[k].s))
                return RECUR_EARG;
        if (meet(o[i].s, ws))
            return RECUR_EARG;
    }
    for (const Buf &b : ins)
        if (meet(ws, b.s))
            return RECUR_EARG;
    return RECUR_OK;
}

bool bad_ld(const recur_config *c, int64_t ld) { return ld < c->dim || ld > INT32_MAX; }

Buf strided(const recur_config *c, const void *p, int64_t ld, int64_t T)
{
    const uint64_t e = size_of(c->dtype);
    return Buf{Span{p, (uint64_t)c->dim * e, (uint64_t)T, (uint64_t)ld * e}, e, true};
}
Buf rows_of(const recur_config *c, const void *p, int64_t T)
{
    const uint64_t e = size_of(c->dtype);
    return Buf{Span{p, (uint64_t)T * c->dim * e}, e, true};
}
Buf states_of(const recur_config *c, const void *p, int64_t n, bool needed = false)
{
    return Buf{Span{p, (uint64_t)n * c->dim * 4}, 4, needed};
}

int check_call(const recur_config *cfg, int pass, const void *ws, uint64_t ws_bytes, const recur_inputs *in,
               const int32_t *offsets, int64_t n, int64_t T)
{
    const int rc = check_config(cfg);
    if (rc)
        return rc;
    if (!in || !ws)
        return RECUR_ENULL;
    if ((uintptr_t)ws % kAlign || (uintptr_t)offsets % 4)
        return RECUR_EALIGN;
    if (T < 0 || T > cfg->max_tokens || n < 0 || n > (int64_t(1) << 24) || (!offsets && n != 1) ||
        bad_ld(cfg, in->ldx) || bad_ld(cfg, in->ldr) || bad_ld(cfg, in->ldi) || ws_bytes < ws_need(cfg, pass))
        return RECUR_ESIZE;
    const int64_t count = chunks(pass, T);   // a launch counts its threads in 32 bits
    return count * columns(cfg->dim, per_lane(cfg, pass, count)) < (int64_t(1) << 23) ? RECUR_OK : RECUR_ESIZE;
}

Args base(const recur_config *c, const recur_inputs *in, const float *lam, int64_t T)
{
    const int64_t e = (int64_t)size_of(c->dtype);
    Args a{};
    a.x = (const uint8_t *)in->x;
    a.r = (const uint8_t *)in->r;
    a.i = (const uint8_t *)in->i;
    a.ldx = in->ldx * e;
    a.ldr = in->ldr * e;
    a.ldi = in->ldi * e;
    a.lam = lam;
    a.T = T;
    a.D = c->dim;
    a.c = c->c;
    a.accum = (c->options & RECUR_OPT_ACCUM) != 0;
    return a;
}

void place_words(const recur_config *c, Args &a, int pass, void *ws)
{
    uint8_t *p = (uint8_t *)ws;
    const int64_t n = chunks(pass, a.T);
    a.per = per_lane(c, pass, n);
    a.columns = (int)columns(a.D, a.per);
    a.chunks = (int)n;
    a.alone = n <= 1;
    a.words = (int64_t)words_of(a.D, n);
    a.tickets = (uint32_t *)p;
    p += ticket_bytes(a.D);
    a.sums = (uint64_t *)p;
    a.states = a.sums + n * (int64_t)row_words(a.D);
    a.part = (float *)(p + align_up((uint64_t)a.words * 8));
}

// What has to be done before the chunks; states without rows: out = in.
void clear(const Args &a, const float *in, float *out, hipStream_t s)
{
    if (a.alone && !(out && (a.offsets || a.T == 0)))
        return;
    const int64_t words = a.alone ? 1 : a.words;
    const unsigned grid = (unsigned)std::min<int64_t>(2048, std::max((words + 2047) / 2048, out ? a.n : 1));
    clear_kernel<<<grid, 256, 0, s>>>(a, in, out);
}

int done() { return hipGetLastError() == hipSuccess ? RECUR_OK : RECUR_EHIP; }

}   // namespace
}   // namespace recur

using namespace recur;

extern "C" {

int recur_abi_version(void) { return RECUR_ABI_VERSION; }

const char *recur_status_string(int status)
{
    switch (status) {
    case RECUR_OK: return "ok";
    case RECUR_ENULL: return "a required pointer is NULL";
    case RECUR_EALIGN: return "a pointer is misaligned";
    case RECUR_ECONFIG: return "invalid config";
    case RECUR_ESIZE: return "size out of range or workspace too small";
    case RECUR_EARG: return "buffers overlap, or an unknown pass";
    case RECUR_EHIP: return "HIP runtime error";
    default: return "unknown status";
    }
}

int recur_config_check(const recur_config *cfg) { return check_config(cfg); }

int recur_workspace_bytes(const recur_config *cfg, int pass, uint64_t *bytes)
{
    const int rc = check_config(cfg);
    if (rc)
        return rc;
    if (!bytes)
        return RECUR_ENULL;
    if (pass != RECUR_PASS_FWD && pass != RECUR_PASS_BWD)
        return RECUR_EARG;
    *bytes = ws_need(cfg, pass);
    return RECUR_OK;
}

int recur_saved_bytes(const recur_config *cfg, int64_t T, uint64_t *bytes)
{
    const int rc = check_config(cfg);
    if (rc)
        return rc;
    if (!bytes)
        return RECUR_ENULL;
    if (T < 0 || T > cfg->max_tokens)
        return RECUR_ESIZE;
    *bytes = (uint64_t)saved_rows(T) * cfg->dim * 4;
    return RECUR_OK;
}

int recur_fwd(const recur_config *cfg, void *ws, uint64_t ws_bytes, const recur_inputs *in, const float *lam,
              const int32_t *offsets, int64_t n, const float *h0, int64_t T, void *y, float *hT, float *saved,
              void *stream)
{
    int rc = check_call(cfg, RECUR_PASS_FWD, ws, ws_bytes, in, offsets, n, T);
    if (rc)
        return rc;
    if ((rc = check({strided(cfg, in->x, in->ldx, T), strided(cfg, in->r, in->ldr, T), strided(cfg, in->i, in->ldi, T),
                     states_of(cfg, lam, 1, true), Buf{Span{offsets, offsets ? 4 * ((uint64_t)n + 1) : 0}, 4, false},
                     states_of(cfg, h0, n)},
                    {rows_of(cfg, y, T), states_of(cfg, hT, n), states_of(cfg, saved, saved_rows(T))}, Span{ws, ws_bytes})))
        return rc;
    if (n == 0 || (T == 0 && !hT))
        return RECUR_OK;
    Args a = base(cfg, in, lam, T);
    a.offsets = offsets;
    a.n = n;
    a.h0 = h0;
    a.y = (uint8_t *)y;
    a.hT = hT;
    a.saved = saved;
    place_words(cfg, a, RECUR_PASS_FWD, ws);
    hipStream_t s = (hipStream_t)stream;
    clear(a, h0, hT, s);
    if (T) {
        const bool f32 = cfg->dtype == RECUR_DTYPE_F32, one = a.per == 1;
        const int w = waves(RECUR_PASS_FWD, T);
        auto k = w == kManyWaves ? (f32 ? fwd_kernel<4, 1, kManyWaves> : fwd_kernel<2, 1, kManyWaves>)
                 : f32           ? (one ? fwd_kernel<4, 1, kWaves> : fwd_kernel<4, 2, kWaves>)
                                 : (one ? fwd_kernel<2, 1, kWaves> : fwd_kernel<2, 2, kWaves>);
        k<<<(unsigned)(chunks(RECUR_PASS_FWD, T) * a.columns), w * 64, 0, s>>>(a);
    }
    return done();
}

int recur_bwd(const recur_config *cfg, void *ws, uint64_t ws_bytes, const recur_inputs *in, const float *lam,
              const int32_t *offsets, int64_t n, const float *h0, const float *saved, const void *dy,
              const float *dhT, int64_t T, const recur_grads *out, float *dlam, float *dh0, void *stream)
{
    int rc = check_call(cfg, RECUR_PASS_BWD, ws, ws_bytes, in, offsets, n, T);
    if (rc)
        return rc;
    if (!out)
        return RECUR_ENULL;
    if (bad_ld(cfg, out->lddx) || bad_ld(cfg, out->lddr) || bad_ld(cfg, out->lddi))
        return RECUR_ESIZE;
    if ((rc = check({strided(cfg, in->x, in->ldx, T), strided(cfg, in->r, in->ldr, T), strided(cfg, in->i, in->ldi, T),
                     states_of(cfg, lam, 1, true), Buf{Span{offsets, offsets ? 4 * ((uint64_t)n + 1) : 0}, 4, false},
                     states_of(cfg, h0, n), states_of(cfg, saved, saved_rows(T), true), rows_of(cfg, dy, T),
                     states_of(cfg, dhT, n)},
                    {strided(cfg, out->dx, out->lddx, T), strided(cfg, out->dr, out->lddr, T),
                     strided(cfg, out->di, out->lddi, T), states_of(cfg, dlam, 1, true), states_of(cfg, dh0, n)},
                    Span{ws, ws_bytes})))
        return rc;
    Args a = base(cfg, in, lam, T);
    a.offsets = offsets;
    a.n = n;
    a.h0 = h0;
    a.saved = const_cast<float *>(saved);
    a.dy = (const uint8_t *)dy;
    a.dhT = dhT;
    const int64_t e = (int64_t)size_of(cfg->dtype);
    a.dx = (uint8_t *)out->dx;
    a.dr = (uint8_t *)out->dr;
    a.di = (uint8_t *)out->di;
    a.lddx = out->lddx * e;
    a.lddr = out->lddr * e;
    a.lddi = out->lddi * e;
    a.dlam = dlam;
    a.dh0 = dh0;
    if (n == 0)   // no sequence: nothing but dlam
        a.T = T = 0;
    if (T == 0 && a.accum && !dh0)
        return RECUR_OK;
    place_words(cfg, a, RECUR_PASS_BWD, ws);
    hipStream_t s = (hipStream_t)stream;
    clear(a, dhT, dh0, s);
    if (T) {
        const bool f32 = cfg->dtype == RECUR_DTYPE_F32, one = a.per == 1;
        const int w = waves(RECUR_PASS_BWD, T);
        auto k = w == kManyWaves ? (f32 ? bwd_kernel<4, 1, kManyWaves> : bwd_kernel<2, 1, kManyWaves>)
                 : f32           ? bwd_kernel<4, 1, kWaves>
                                 : (one ? bwd_kernel<2, 1, kWaves> : bwd_kernel<2, 2, kWaves>);
        k<<<(unsigned)(chunks(RECUR_PASS_BWD, T) * a.columns), w * 64, 0, s>>>(a);
    }
    if (T ? !a.alone : !a.accum)
        dlam_kernel<<<(cfg->dim + 15) / 16, 1024, 0, s>>>(a);
    return done();
}

int recur_step(const recur_config *cfg, const recur_inputs *in, const float *lam, float *state, int64_t states,
               const int32_t *slots, int64_t n, void *y, void *stream)
{
    int rc = check_config(cfg);
    if (rc)
        return rc;
    if (!in)
        return RECUR_ENULL;
    if (n < 0 || n > (int64_t(1) << 16) || states < 0 || states > INT32_MAX || (!slots && states < n) ||
        bad_ld(cfg, in->ldx) || bad_ld(cfg, in->ldr) || bad_ld(cfg, in->ldi))
        return RECUR_ESIZE;
    if ((rc = check({strided(cfg, in->x, in->ldx, n), strided(cfg, in->r, in->ldr, n), strided(cfg, in->i, in->ldi, n),
                     states_of(cfg, lam, 1, true), Buf{Span{slots, slots ? 4 * (uint64_t)n : 0}, 4, false}},
                    {rows_of(cfg, y, n), states_of(cfg, state, states, true)}, Span{nullptr, 0})))
        return rc;
    if (n == 0)
        return RECUR_OK;
    Args a = base(cfg, in, lam, n);
    a.y = (uint8_t *)y;
    a.n = n;
    const bool f32 = cfg->dtype == RECUR_DTYPE_F32;
    a.per = a.D % 2 ? 1 : per_lane(a.D, n);
    a.columns = (int)columns(a.D, a.per);
    const bool one = a.per == 1;
    auto k = f32 ? (one ? step_kernel<4, 1> : step_kernel<4, 2>) : (one ? step_kernel<2, 1> : step_kernel<2, 2>);
    k<<<(unsigned)((n * a.columns + 3) / 4), 256, 0, (hipStream_t)stream>>>(a, state, (int)states, slots, (int)n);
    return done();
}

}   // extern "C"
