// attn_shared.cuh -- the plan of tree-verify attention over shared prefixes.
//
// Sequences of a group have their first `used` pages in common.  Those pages are one
// key segment for all rows of the group (nodes of consecutive sequences, times the
// heads of a KV head), cut into row blocks of at most kRowsMax rows; what a
// sequence has for itself (its other pages and, as a last page, its tree) is a
// segment of its own rows, cut into row groups as in the windowed attention.  Two
// pages make a key tile.  The plan cuts both kinds into pieces, a list for
// each CTA; a piece that does not hold all keys of its rows leaves a partial
// (O, max, sum) in its slot of the workspace, and the merge joins a row's slots.
#pragma once

#include "internal.cuh"

namespace lucetree {
namespace shr {

constexpr int kMagic = 0x6c745370;
constexpr int kMaxParts = 4;  // a CTA's fair share of tiles is cut into at most so many shared pieces
constexpr int kMaxCtas = 1024;

struct Dims {
    int B, N, Hq, Hkv, G, D, groups;
    int C;          // CTAs
    RowGroups own;  // of a sequence's rows
    int NPG, RG;    // of a shared row block: nodes (of any sequences of the group), rows
    __host__ __device__ int segs() const { return B * Hkv * own.NG; }
    __host__ __device__ long long max_items() const {
        return (long long)kMaxParts * C + (long long)Hkv * ((long long)B * N / NPG + groups);
    }
    __host__ __device__ long long max_own() const { return (long long)C + (long long)B * Hkv * own.NG; }
};

inline Dims make_dims(int B, int N, int Hq, int Hkv, int D, int groups, int ctas) {
    Dims d;
    d.B = B; d.N = N; d.Hq = Hq; d.Hkv = Hkv; d.G = Hq / Hkv; d.D = D; d.groups = groups; d.C = ctas;
    d.own = make_row_groups(N, d.G);
    // row blocks of equal size for a group of the mean number of sequences
    const long long nodes = (long long)((B + groups - 1) / groups) * N;
    const long long cap = kRowsMax / d.G, blocks = (nodes + cap - 1) / cap;
    d.NPG = (int)((nodes + blocks - 1) / blocks);
    d.RG = d.NPG * d.G;
    return d;
}

// What a CTA does at a time: tiles [ta, te) of a segment's list of pages for some rows.
struct Piece {
    int b, g;           // sequence whose table row names the pages, KV head
    int node0, nodes;   // rows: nodes [node0, node0 + nodes) of all sequences' nodes
    int page0, vp;      // the segment's pages: vp of them from column page0 on, then the tree's if own
    int ta, te;
    int keys;           // committed keys from the first of page0 on
    int slot;           // of its kind's partial sums
    int own;            // a sequence's own segment (else a group's)
    int reread;         // other row blocks read the same keys
};
static_assert(sizeof(Piece) == 48, "three 16-byte words");

struct Cta {
    int own0, owns;  // its own-segment pieces [own0, own0 + owns)
    int tiles;       // of all its pieces
    int items;       // shared pieces: cta, cta + C, ..
};

struct Group {
    int used;   // pages that are read once for the group
    int base;   // first shared piece (and slot)
    int parts;  // pieces of a row block and KV head
    int blocks; // row blocks
};

struct Seq {
    int group, first;  // its group and that one's first sequence
    int L, used, off;  // committed length, pages read with the group, flat number of its first own tile
};

struct Seg {
    int first, count;  // its pieces, which are its slots too; count < 0: one piece that holds all its rows' keys
};

struct Head {
    int magic, B, N, Hq, Hkv, D, groups, C, max_pages, num_pages;
    int parts;  // shared pieces
    int pad[5];
};

struct Plan {  // a plan's parts in its buffer
    Head* head;
    Cta* cta;
    Group* grp;
    Seq* seq;
    Seg* seg;
    int* lcp;      // pages that a row has in common with its group's first
    Piece* item;   // shared pieces, [part][row block] of each KV head of each group
    Piece* piece;  // own pieces
};

__host__ __device__ inline size_t up16(size_t n) { return (n + 15) / 16 * 16; }

__host__ __device__ inline size_t plan_bytes(const Dims& d, Plan* p, void* at) {
    char* base = reinterpret_cast<char*>(at);
    size_t n = 0;
    auto take = [&](size_t bytes) {
        char* x = base + n;
        n += up16(bytes);
        return x;
    };
    Plan q;
    q.head = reinterpret_cast<Head*>(take(sizeof(Head)));
    q.cta = reinterpret_cast<Cta*>(take(sizeof(Cta) * (size_t)d.C));
    q.grp = reinterpret_cast<Group*>(take(sizeof(Group) * (size_t)d.groups));
    q.seq = reinterpret_cast<Seq*>(take(sizeof(Seq) * (size_t)d.B));
    q.seg = reinterpret_cast<Seg*>(take(sizeof(Seg) * (size_t)d.segs()));
    q.lcp = reinterpret_cast<int*>(take(sizeof(int) * (size_t)d.B));
    q.item = reinterpret_cast<Piece*>(take(sizeof(Piece) * (size_t)d.max_items()));
    q.piece = reinterpret_cast<Piece*>(take(sizeof(Piece) * (size_t)d.max_own()));
    if (p) *p = q;
    return n;
}

// Floats of a slot of partial sums: O [rows][D], max [rows], sum [rows].
__host__ __device__ inline size_t slot_floats(int rows, int D) { return ((size_t)rows * (D + 2) + 63) / 64 * 64; }

__host__ __device__ inline size_t workspace_bytes(const Dims& d) {
    return sizeof(float) * ((size_t)d.max_items() * slot_floats(d.RG, d.D) + (size_t)d.max_own() * slot_floats(d.own.RG, d.D));
}

struct Launch {
    lucetree_attn_args a;  // a.out is not used
    Dims d;
    Plan plan;
    float* shared_ws;      // slots of shared pieces
    float* own_ws;         // slots of own pieces
    float scale_log2;
    int out_dtype;         // LUCETREE_F32 or a.dtype
    void* out;
};

// Whether the plan was made for a call of these sizes.
__device__ inline bool plan_fits(const Launch& W) {
    const Head h = *W.plan.head;
    return h.magic == kMagic && h.B == W.d.B && h.N == W.d.N && h.Hq == W.d.Hq && h.Hkv == W.d.Hkv && h.D == W.d.D &&
           h.groups == W.d.groups && h.C == W.d.C && h.max_pages == W.a.max_pages_per_seq &&
           h.num_pages == W.a.num_pages;
}

cudaError_t launch_shared_plan(const lucetree_shared_plan_args& a, const Dims& d, cudaStream_t stream);
cudaError_t launch_shared_merge(const Launch& W, cudaStream_t stream);

}  // namespace shr
}  // namespace lucetree
