// The gated linear recurrence (include/recur.h).
//
// A block takes a chunk of 64 positions of 128 channels: 8 wavefronts of 8 positions,
// a lane two channels.  A stretch of positions is h -> A h + H, so stretches join:
// positions in registers, wavefronts through LDS, chunks through words of the
// workspace that say by themselves when they are there (state_before).  Every input
// is read once and every output written once.
#include <algorithm>
#include <initializer_list>

#include "recur_dev.hpp"
#include "spans.hpp"

namespace recur {
namespace {

using spans::meet;
using spans::Span;

constexpr uint64_t kAlign = 256;
constexpr int kThreads = kWaves * 64;

// Where sequences begin and end among a chunk's positions.
struct Marks {
    unsigned long long starts, ends;
    int start_of[kChunk], end_of[kChunk];   // the sequence, where the bit is set
};

// A wavefront's view of them: bit k is its position k.
struct Bits {
    uint32_t starts, ends, inside;
};

// All threads of the block.  The sequences that can matter: those from the last
// probe that begins in front of t0 to the first that begins behind the chunk.
__device__ void find_marks(const Args &a, int64_t t0, Marks *m)
{
    __shared__ int from, to;
    if (threadIdx.x == 0) {
        m->starts = m->ends = 0;
        from = 0;
        to = (int)a.n;
    }
    __syncthreads();
    if (a.n > 4 * kThreads) {
        const int64_t step = (a.n + kThreads - 1) / kThreads, at = threadIdx.x * step;
        if (at < a.n) {
            const int32_t v = a.offsets[at];
            if (v < t0)
                atomicMax(&from, (int)at);
            if (v > t0 + kChunk)
                atomicMin(&to, (int)at);
        }
        __syncthreads();
    }
    for (int s = from + (int)threadIdx.x; s < to; s += kThreads) {
        const int64_t b = a.offsets[s], e = a.offsets[s + 1];
        if (b >= e)
            continue;
        if (b >= t0 && b < t0 + kChunk) {
            atomicOr(&m->starts, 1ull << (b - t0));
            m->start_of[b - t0] = s;
        }
        if (e > t0 && e <= t0 + kChunk) {
            atomicOr(&m->ends, 1ull << (e - 1 - t0));
            m->end_of[e - 1 - t0] = s;
        }
    }
    __syncthreads();
}

// The block's chunk, and its place side by side.  A block that waits for others
// takes its place when it begins to run, in the order in which chunks depend on
// one another: whoever it waits for has begun before it.
__device__ __forceinline__ void place(const Args &a, int &chunk, int &column)
{
    __shared__ uint32_t ticket;
    chunk = 0;
    column = blockIdx.x;
    if (a.chunks > 1) {
        if (threadIdx.x == 0)
            ticket = atomicAdd(a.ticket, 1u);
        __syncthreads();
        chunk = (int)(ticket / (uint32_t)a.columns);
        column = (int)(ticket % (uint32_t)a.columns);
    }
}

// The rows that belong to a sequence.
__device__ __forceinline__ void rows_of_sequences(const Args &a, int64_t &lo, int64_t &hi)
{
    lo = a.offsets ? max((int64_t)0, (int64_t)a.offsets[0]) : 0;
    hi = a.offsets ? min(a.T, (int64_t)a.offsets[a.n]) : a.T;
}

__device__ __forceinline__ Bits bits_of(const Args &a, const Marks *m, int64_t t0, int64_t lo, int64_t hi, int wave)
{
    Bits b;
    const int64_t t = t0 + wave * kSteps;
    if (a.offsets) {
        b.starts = (uint32_t)(m->starts >> (wave * kSteps)) & ((1u << kSteps) - 1);
        b.ends = (uint32_t)(m->ends >> (wave * kSteps)) & ((1u << kSteps) - 1);
    } else {
        b.starts = t == 0 ? 1u : 0u;
        b.ends = hi > t && hi <= t + kSteps ? 1u << (hi - 1 - t) : 0u;
    }
    b.inside = 0;
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
        b.inside |= (t + k >= lo && t + k < hi ? 1u : 0u) << k;
    b.starts = __builtin_amdgcn_readfirstlane(b.starts & b.inside);
    b.ends = __builtin_amdgcn_readfirstlane(b.ends & b.inside);
    b.inside = __builtin_amdgcn_readfirstlane(b.inside);
    return b;
}

template <int V>
struct Shared {
    Span1 waves[kWaves][V][64];   // each wavefront's stretch
    Span1 before[kWaves][V][64];  // stretches of the chunks before, kGroup / kWaves a wavefront
    float state[V][64];           // the state in front of the group of chunks
    Marks marks;
};

// The state in front of the block's chunk; `index` counts chunks in the order in
// which they depend on one another.  own: the wavefront's stretch, `order` its
// place in the block in that order.
//
// Every chunk says what it does to a state (sums) as soon as it knows it, without
// waiting for anyone; the last chunk of a group of kGroup says what state it leaves
// (states).  A chunk takes the state in front of its group and goes through the
// group's earlier chunks, always in the same order, so that results do not depend
// on who came first.  A wait ends: who is waited for has begun to run (place), and
// waits itself only for chunks in front of it; should one never answer, the values
// become NaN after a bounded number of polls.
template <int V>
__device__ __forceinline__ void state_before(const Args &a, Shared<V> &sh, int index, int wave, int order, int lane,
                                             int j, const Span1 (&own)[V], float (&h)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v)
        sh.waves[order][v][lane] = own[v];
    __syncthreads();
    if (a.chunks > 1) {
        Span1 all[V];
        if (wave == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                all[v] = sh.waves[0][v][lane];
#pragma unroll
                for (int w = 1; w < kWaves; ++w)
                    all[v] = join(all[v], sh.waves[w][v][lane]);
                publish(&a.sums[(int64_t)index * a.D + j + v], word(all[v]));
            }
        }
        const int group = index / kGroup, place = index % kGroup, per = kGroup / kWaves;
        uint64_t w[per][V], s[V];
        const bool first = wave == kWaves - 1 && group > 0;
        for (int polls = 0; polls < (1 << 20); ++polls) {
            bool there = true;
#pragma unroll
            for (int i = 0; i < per; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    w[i][v] = 0;
                    if (wave * per + i < place)
                        w[i][v] = peek(&a.sums[((int64_t)group * kGroup + wave * per + i) * a.D + j + v]);
                }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[v] = 0;
                if (first)
                    s[v] = peek(&a.states[(int64_t)group * a.D + j + v]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                there = there && s[v] != kNone;
#pragma unroll
                for (int i = 0; i < per; ++i)
                    there = there && w[i][v] != kNone;
            }
            if (__all(there))
                break;
            __builtin_amdgcn_s_sleep(1);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            Span1 p{1.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < per; ++i)
                if (wave * per + i < place)
                    p = join(p, span(w[i][v]));
            sh.before[wave][v][lane] = p;
            if (wave == kWaves - 1)
                sh.state[v][lane] = group > 0 ? span(s[v]).H : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = sh.state[v][lane];
#pragma unroll
            for (int i = 0; i < kWaves; ++i)
                h[v] = through(sh.before[i][v][lane], h[v]);
            if (wave == 0 && place == kGroup - 1 && index + 1 < a.chunks)
                publish(&a.states[(int64_t)(group + 1) * a.D + j + v], word(Span1{1.0f, through(all[v], h[v])}));
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            h[v] = 0.0f;
    }
}

// Clears the words that blocks wait for, and gives sequences without rows their
// states: out = in (or 0).
__global__ __launch_bounds__(256) void clear_kernel(Args a, const float *in, float *out)
{
    const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    if (a.chunks > 1) {
        const int64_t words = (int64_t)(a.chunks + a.chunks / kGroup + 1) * a.D;   // sums, then states
        for (int64_t k = first; k < words; k += step)
            a.sums[k] = kNone;
        if (first == 0)
            *a.ticket = 0;
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

template <int E, int V>
__global__ __launch_bounds__(kThreads) void fwd_kernel(Args a)
{
    __shared__ Shared<V> sh;
    int chunk, column;
    place(a, chunk, column);
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    // lanes past the last channels take those again: the same loads, values and stores
    const int j = min((column * 64 + lane) * V, a.D - V);
    const uint32_t off = (uint32_t)j * E;   // behind a row's address, which is the same for all lanes
    const int64_t t0 = (int64_t)chunk * kChunk, t = t0 + wave * kSteps;
    int64_t lo, hi;
    rows_of_sequences(a, lo, hi);
    if (t0 >= hi)
        return;   // nor does any chunk behind it ask
    Raw<E, V> x[kSteps], r[kSteps], i[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        const int64_t row = min(t + k, a.T - 1);
        r[k] = load<E, V>(a.r + row * a.ldr + off);
        i[k] = load<E, V>(a.i + row * a.ldi + off);
        x[k] = load<E, V>(a.x + row * a.ldx + off);
    }
    float rate[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        rate[v] = decay(a.lam[j + v], a.c);
    if (a.offsets)
        find_marks(a, t0, &sh.marks);
    const Bits bits = bits_of(a, &sh.marks, t0, lo, hi, wave);
    float av[kSteps][V], u[kSteps][V];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        float xf[V], rf[V], gf[V];
        unpack<E, V>(x[k], xf);
        unpack<E, V>(r[k], rf);
        unpack<E, V>(i[k], gf);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Gates q = gates(rf[v], gf[v], rate[v]);
            av[k][v] = q.a;
            u[k][v] = q.m * q.g * xf[v];
        }
    }
    Span1 own[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        own[v] = Span1{1.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        if (!(bits.inside >> k & 1)) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                av[k][v] = 1.0f;
                u[k][v] = 0.0f;
            }
        }
        if (bits.starts >> k & 1) {
            if (a.h0) {
                const int64_t s = a.offsets ? sh.marks.start_of[wave * kSteps + k] : 0;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    u[k][v] = __builtin_fmaf(av[k][v], a.h0[s * a.D + j + v], u[k][v]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
                own[v].H = u[k][v];
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                own[v].A *= av[k][v];
                own[v].H = __builtin_fmaf(av[k][v], own[v].H, u[k][v]);
            }
        }
    }
    if (bits.starts) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            own[v].A = -1.0f;
    }
    float h[V];
    state_before<V>(a, sh, chunk, wave, wave, lane, j, own, h);
    if (a.saved && wave == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            a.saved[(int64_t)chunk * a.D + j + v] = h[v];
    }
    for (int w = 0; w < wave; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v)
            h[v] = through(sh.waves[w][v][lane], h[v]);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            h[v] = bits.starts >> k & 1 ? u[k][v] : __builtin_fmaf(av[k][v], h[v], u[k][v]);
        if (bits.inside >> k & 1)
            store<E, V>(a.y + (t + k) * a.D * E + off, h);
        if (a.hT && (bits.ends >> k & 1)) {
            const int64_t s = a.offsets ? sh.marks.end_of[wave * kSteps + k] : 0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                a.hT[s * a.D + j + v] = h[v];
        }
    }
}

// Chunks from the last to the first.  The states come from the saved one, forward
// through the chunk; with them and the gates every output is G_t times a number of
// its position: dx c1, di c2, dr cr, and rho dz (of dlam) cl.  G in turn runs
// backwards, what a position hands on being a_t G_t.
template <int E, int V>
__global__ __launch_bounds__(kThreads) void bwd_kernel(Args a)
{
    __shared__ Shared<V> sh;
    int index, column;
    place(a, index, column);
    const int chunk = a.chunks - 1 - index;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int j = min((column * 64 + lane) * V, a.D - V);
    const uint32_t off = (uint32_t)j * E;   // behind a row's address, which is the same for all lanes
    const int64_t t0 = (int64_t)chunk * kChunk, t = t0 + wave * kSteps;
    Raw<E, V> x[kSteps], r[kSteps], i[kSteps], d[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        const int64_t row = min(t + k, a.T - 1);
        r[k] = load<E, V>(a.r + row * a.ldr + off);
        i[k] = load<E, V>(a.i + row * a.ldi + off);
        x[k] = load<E, V>(a.x + row * a.ldx + off);
        d[k] = load<E, V>(a.dy + row * a.D * E + off);
    }
    float rate[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        rate[v] = decay(a.lam[j + v], a.c);
        h[v] = a.saved[(int64_t)chunk * a.D + j + v];
    }
    int64_t lo, hi;
    rows_of_sequences(a, lo, hi);
    if (a.offsets)
        find_marks(a, t0, &sh.marks);
    const Bits bits = bits_of(a, &sh.marks, t0, lo, hi, wave);
    float av[kSteps][V], c1[kSteps][V], c2[kSteps][V], cr[kSteps][V], cl[kSteps][V], u[kSteps][V], c3[kSteps][V];
    Span1 own[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        own[v] = Span1{1.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        float xf[V], rf[V], gf[V];
        unpack<E, V>(x[k], xf);
        unpack<E, V>(r[k], rf);
        unpack<E, V>(i[k], gf);
        const bool start = bits.starts >> k & 1, inside = bits.inside >> k & 1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Gates q = gates(rf[v], gf[v], rate[v]);
            av[k][v] = inside ? q.a : 1.0f;
            c1[k][v] = q.m * q.g;
            u[k][v] = inside ? c1[k][v] * xf[v] : 0.0f;
            c2[k][v] = u[k][v] * q.g_rest;
            cl[k][v] = q.rho;
            cr[k][v] = rate[v] * q.rho * q.rho_rest;
            c3[k][v] = q.m > 0.0f ? q.g * xf[v] * (q.a * q.a * __builtin_amdgcn_rcpf(q.m)) : 0.0f;
        }
        if (start && a.h0) {
            const int64_t s = a.offsets ? sh.marks.start_of[wave * kSteps + k] : 0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                u[k][v] = __builtin_fmaf(av[k][v], a.h0[s * a.D + j + v], u[k][v]);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            own[v].A *= av[k][v];
            own[v].H = start ? u[k][v] : __builtin_fmaf(av[k][v], own[v].H, u[k][v]);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            here(c1[k][v]);
            here(c2[k][v]);
            here(c3[k][v]);
            here(cl[k][v]);
            here(cr[k][v]);
        }
    }
    // h_{t-1}, and what it makes of the numbers above
#pragma unroll
    for (int v = 0; v < V; ++v)
        sh.before[wave][v][lane] = Span1{bits.starts ? -1.0f : own[v].A, own[v].H};
    __syncthreads();
    for (int w = 0; w < wave; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v)
            h[v] = through(sh.before[w][v][lane], h[v]);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        const bool start = bits.starts >> k & 1;
        if (start) {
            const int64_t s = a.offsets ? sh.marks.start_of[wave * kSteps + k] : 0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                h[v] = a.h0 ? a.h0[s * a.D + j + v] : 0.0f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float z = __builtin_fmaf(av[k][v], h[v], -c3[k][v]);   // dz / G
            cr[k][v] *= z;
            cl[k][v] *= z;
            here(cr[k][v]);
            here(cl[k][v]);
            h[v] = start ? u[k][v] : __builtin_fmaf(av[k][v], h[v], u[k][v]);
        }
    }
    // the same backwards: what reaches the stretch from behind goes to A in + H
    Span1 back[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        back[v] = Span1{bits.ends ? -1.0f : own[v].A, 0.0f};
    float df[kSteps][V];
#pragma unroll
    for (int k = kSteps - 1; k >= 0; --k) {
        unpack<E, V>(d[k], df[k]);
        const bool end = bits.ends >> k & 1, inside = bits.inside >> k & 1;
        if (end) {
            const int64_t s = a.offsets ? sh.marks.end_of[wave * kSteps + k] : 0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                back[v].H = a.dhT ? a.dhT[s * a.D + j + v] : 0.0f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            df[k][v] = inside ? df[k][v] : 0.0f;
            if (end)
                df[k][v] += back[v].H;   // kept: the second walk then begins at 0 here
            back[v].H = av[k][v] * (end ? df[k][v] : df[k][v] + back[v].H);
        }
    }
    float in[V], acc[V];
    state_before<V>(a, sh, index, wave, kWaves - 1 - wave, lane, j, back, in);
    for (int w = 0; w < kWaves - 1 - wave; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v)
            in[v] = through(sh.waves[w][v][lane], in[v]);
#pragma unroll
    for (int v = 0; v < V; ++v)
        acc[v] = 0.0f;
#pragma unroll
    for (int k = kSteps - 1; k >= 0; --k) {
        const bool end = bits.ends >> k & 1;
        float dx[V], di[V], dr[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float G = end ? df[k][v] : df[k][v] + in[v];
            in[v] = av[k][v] * G;
            dx[v] = G * c1[k][v];
            di[v] = G * c2[k][v];
            dr[v] = G * cr[k][v];
            cl[k][v] *= G;
        }
        if (bits.inside >> k & 1) {
            store<E, V>(a.dx + (t + k) * a.lddx + off, dx);
            store<E, V>(a.di + (t + k) * a.lddi + off, di);
            store<E, V>(a.dr + (t + k) * a.lddr + off, dr);
#pragma unroll
            for (int v = 0; v < V; ++v)
                acc[v] += cl[k][v];
        }
        if (a.dh0 && (bits.starts >> k & 1)) {
            const int64_t s = a.offsets ? sh.marks.start_of[wave * kSteps + k] : 0;
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
            for (int w = 1; w < kWaves; ++w)
                s += sh.waves[w][v][lane].A;
            a.part[(int64_t)chunk * a.D + j + v] = s;
        }
    }
}

// dlam from the chunks' parts, in a fixed order: 64 channels a block, 16 threads to
// a channel.
__global__ __launch_bounds__(1024) void dlam_kernel(Args a)
{
    __shared__ float lds[16][64];
    const int c = threadIdx.x % 64, g = threadIdx.x / 64, j = blockIdx.x * 64 + c;
    float s = 0.0f;
    if (j < a.D) {
#pragma unroll 8
        for (int64_t k = g; k < a.chunks; k += 16)
            s += a.part[k * a.D + j];
    }
    lds[g][c] = s;
    __syncthreads();
    if (g != 0 || j >= a.D)
        return;
#pragma unroll
    for (int k = 1; k < 16; ++k)
        s += lds[k][c];
    float sl, rest;
    sigmoid(a.lam[j], sl, rest);
    const float v = alone(-a.c * sl, s);
    a.dlam[j] = a.accum ? a.dlam[j] + v : v;
}

template <int E>
__device__ __forceinline__ float at(const uint8_t *row, int j)
{
    float v[1];
    unpack<E, 1>(load<E, 1>(row + (int64_t)j * E), v);
    return v[0];
}

// A wavefront a row and 64 channels.  Rows of one slot form a chain: its first
// row takes them all, in order.
template <int E>
__global__ __launch_bounds__(64) void step_kernel(Args a, float *state, int64_t states, const int32_t *slots)
{
    const int j = blockIdx.x * 64 + threadIdx.x;
    const int64_t row = blockIdx.y;
    const int64_t slot = slots ? slots[row] : row;
    if (slot < 0 || slot >= states) {
        if (j < a.D)
            store<E, 1>(a.y + (row * a.D + j) * E, {0.0f});
        return;
    }
    if (slots) {
        for (int64_t k = 0; k < row; ++k)
            if (slots[k] == slot)
                return;
    }
    if (j >= a.D)
        return;
    const float k = decay(a.lam[j], a.c);
    float h = state[slot * a.D + j];
    for (int64_t t = row; t < (slots ? a.n : row + 1); ++t) {
        if (slots && slots[t] != slot)
            continue;
        const Gates v = gates(at<E>(a.r + t * a.ldr, j), at<E>(a.i + t * a.ldi, j), k);
        h = __builtin_fmaf(v.a, h, v.m * v.g * at<E>(a.x + t * a.ldx, j));
        store<E, 1>(a.y + (t * a.D + j) * E, {h});
    }
    state[slot * a.D + j] = h;
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

int64_t chunks(int64_t T) { return (T + kChunk - 1) / kChunk; }
uint64_t align_up(uint64_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

// A lane takes two channels; up to 64 channels one, or half the wavefront would
// have none.
int per_lane(int D) { return D <= 64 ? 1 : 2; }
int64_t columns(int D) { return (D + 64 * per_lane(D) - 1) / (64 * per_lane(D)); }

// Workspace: the ticket, the words of chunks and groups, the parts of dlam.
uint64_t words_bytes(int D, int64_t n) { return align_up((uint64_t)(n + n / kGroup + 1) * D * 8); }
uint64_t ws_need(const recur_config *c, int pass)
{
    const int64_t n = chunks(c->max_tokens);
    return kAlign + words_bytes(c->dim, n) + (pass == RECUR_PASS_BWD ? align_up((uint64_t)n * c->dim * 4) : 0);
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
        bad_ld(cfg, in->ldx) || bad_ld(cfg, in->ldr) || bad_ld(cfg, in->ldi) || ws_bytes < ws_need(cfg, pass) ||
        chunks(T) * columns(cfg->dim) >= (int64_t(1) << 23))   // a launch counts its threads in 32 bits
        return RECUR_ESIZE;
    return RECUR_OK;
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
    a.chunks = (int)chunks(T);
    a.columns = (int)columns(c->dim);
    return a;
}

void place_words(Args &a, void *ws)
{
    uint8_t *p = (uint8_t *)ws;
    a.ticket = (uint32_t *)p;
    a.sums = (uint64_t *)(p + kAlign);
    a.states = a.sums + (int64_t)a.chunks * a.D;
    a.part = (float *)(p + kAlign + words_bytes(a.D, a.chunks));
}

// What has to be done before the chunks; states without rows: out = in.
void clear(const Args &a, const float *in, float *out, hipStream_t s)
{
    if (a.chunks <= 1 && !(out && (a.offsets || a.chunks == 0)))
        return;
    const int64_t words = a.chunks > 1 ? (int64_t)(a.chunks + a.chunks / kGroup + 1) * a.D : 1;
    const unsigned grid = (unsigned)std::min<int64_t>(2048, std::max((words + 1023) / 1024, out ? a.n : 1));
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
    *bytes = (uint64_t)chunks(T) * cfg->dim * 4;
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
                    {rows_of(cfg, y, T), states_of(cfg, hT, n), states_of(cfg, saved, chunks(T))}, Span{ws, ws_bytes})))
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
    place_words(a, ws);
    hipStream_t s = (hipStream_t)stream;
    clear(a, h0, hT, s);
    if (T) {
        const bool f32 = cfg->dtype == RECUR_DTYPE_F32, one = per_lane(cfg->dim) == 1;
        auto k = f32 ? (one ? fwd_kernel<4, 1> : fwd_kernel<4, 2>) : (one ? fwd_kernel<2, 1> : fwd_kernel<2, 2>);
        k<<<(unsigned)(a.chunks * (int64_t)a.columns), kThreads, 0, s>>>(a);
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
                     states_of(cfg, h0, n), states_of(cfg, saved, chunks(T), true), rows_of(cfg, dy, T),
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
    if (n == 0) {   // no sequence: nothing but dlam
        a.chunks = 0;
        T = 0;
    }
    if (T == 0 && a.accum && !dh0)
        return RECUR_OK;
    place_words(a, ws);
    hipStream_t s = (hipStream_t)stream;
    clear(a, dhT, dh0, s);
    if (T) {
        const bool f32 = cfg->dtype == RECUR_DTYPE_F32, one = per_lane(cfg->dim) == 1;
        auto k = f32 ? (one ? bwd_kernel<4, 1> : bwd_kernel<4, 2>) : (one ? bwd_kernel<2, 1> : bwd_kernel<2, 2>);
        k<<<(unsigned)(a.chunks * (int64_t)a.columns), kThreads, 0, s>>>(a);
    }
    if (T || !a.accum)
        dlam_kernel<<<(cfg->dim + 63) / 64, 1024, 0, s>>>(a);
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
    if (n < 0 || n > (int64_t(1) << 20) || states < 0 || states > INT32_MAX || (!slots && states < n) ||
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
    const dim3 grid((cfg->dim + 63) / 64, (unsigned)n);
    (cfg->dtype == RECUR_DTYPE_F32 ? step_kernel<4> : step_kernel<2>)<<<grid, 64, 0, (hipStream_t)stream>>>(
        a, state, states, slots);
    return done();
}

}   // extern "C"
