// attn_shared.cuh -- the plan of tree-verify attention over shared prefixes.
//
// Rows (nodes of consecutive sequences of a group, times the query heads of a KV head)
// are taken in blocks of at most 128, or of 256 for a pair of CTAs.  A block's key list is made of 64-key
// pages: the group's common pages, which all of its rows see, then for each of its
// sequences the pages that it has for itself, which that sequence's rows see, and last
// the tree nodes of all its sequences (they follow each other in memory), 64 to a page.  Two pages make a key tile.  In a group without common
// pages to read once, a block holds rows of one sequence.  Blocks have the mean group's size, or,
// in a group that this would cut in far more of them than it needs, its own (blocks_of in the
// plan).  The segments (block, KV
// head) form one flat list of tiles that is cut over the CTAs; a piece that does not
// hold all tiles of its segment leaves partial sums (O, max, sum), which the merge
// joins.
#pragma once

#include "internal.cuh"

namespace lucetree {
namespace shr {

constexpr int kMagic = 0x6c745370;
constexpr int kRows = 128;  // of a CTA: the MMA's M
constexpr int kMaxCtas = 512;

// Kinds of blocks: of a group that shares pages, cut by the mean group's size; of a sequence without common
// pages; of a group that shares pages, cut by its own size.
enum { kMeanCut = 0, kOwnCut = 1, kLargeCut = 2 };

struct Dims {
    int B, N, Hq, Hkv, G, D, groups;
    int pair;      // CTAs of a block: 1, or 2 with half of its nodes each
    int C;         // CTAs, or pairs of CTAs
    int cap;       // nodes of a block at most
    int NPG;       // nodes of a block in a group that shares pages, cut by the mean group
    int NG, NPGo;  // other groups: blocks of a sequence, and their nodes
    __host__ __device__ int block_rows() const { return pair * kRows; }
    // nodes of a block in its first CTA, of each kind
    __host__ __device__ int half(int kind) const {
        return ((kind == kOwnCut ? NPGo : kind == kLargeCut ? cap : NPG) + pair - 1) / pair;
    }
    __host__ __device__ int max_blocks() const { return B * NG; }
    __host__ __device__ int max_segs() const { return B * NG * Hkv; }
    __host__ __device__ long long max_pieces() const { return (long long)C + max_segs(); }
};

// Nodes of a block: as few blocks as hold `nodes`, of equal size; whole sequences of N
// where that takes no block more.
inline int block_nodes(long long nodes, int N, int cap) {
    const long long blocks = (nodes + cap - 1) / cap;
    long long per = (nodes + blocks - 1) / blocks;
    const long long whole = (per + N - 1) / N * N;
    if (whole <= cap) per = whole;
    else if (cap >= N && (nodes + cap / N * N - 1) / (cap / N * N) <= blocks) per = cap / N * N;
    return (int)per;
}

inline Dims make_dims(int B, int N, int Hq, int Hkv, int D, int groups, int ctas) {
    Dims d;
    d.B = B; d.N = N; d.Hq = Hq; d.Hkv = Hkv; d.G = Hq / Hkv; d.D = D; d.groups = groups;
    // Pairs where the mean group's rows are more than one CTA's: a pair reads keys once for twice
    // the rows.
    const long long nodes = (long long)((B + groups - 1) / groups) * N;
    d.pair = ctas >= 2 && nodes * d.G > kRows ? 2 : 1;
    d.C = ctas / d.pair;
    const int cap = d.cap = kRows / d.G * d.pair;
    d.NPG = block_nodes(nodes, N, cap);
    d.NG = (N + cap - 1) / cap;
    d.NPGo = (N + d.NG - 1) / d.NG;
    d.NG = (N + d.NPGo - 1) / d.NPGo;
    return d;
}

// A block of rows and its key list.
struct Block {
    int group;
    int b0, seqs;      // its sequences
    int node0, nodes;  // its rows' nodes, of all sequences' nodes
    int used;          // common pages
    int vp;            // pages of the key list
    int pre;           // weight of the blocks before it
};
static_assert(sizeof(Block) == 32, "two 16-byte words");

// What a CTA does at a time: tiles [ta, te) of a segment.
struct Piece {
    int b0, seqs, node0, nodes;  // of its block
    int used, vp;
    int ta, te;
    int g;
    int slot;    // row of the partial sums, -1: all tiles
    int own;     // rows of a sequence without common pages
    int how;     // bit 0: other blocks read most of its pages too; bit 1: its group is cut by its own size
    __device__ int kind() const { return own ? kOwnCut : how & 2; }
};
static_assert(sizeof(Piece) == 48, "three 16-byte words");

// A segment that several CTAs have tiles of, in the place of the first of them.
struct Split {
    int count;         // CTAs, 0: none begins here
    int row;           // the first one's partial sums; the others' follow block_rows() apart
    int node0, rows;   // its rows: those of nodes from node0 on ...
    int g;             // ... and of this KV head
    int pad[3];
};
static_assert(sizeof(Split) == 32, "two 16-byte words");

// A CTA's pieces: its first one stands in its own place r, where it can be fetched with this record,
// the others from `next` on (each begins its segment s, and stands in place C + s).
struct Cta {
    int next, pieces, tiles, pad;
};

struct Group {
    int used;     // pages that are read once for the group
    int block0;   // its first block
    int blocks;
    int seq0, n;  // its first sequence, and how many
};

struct Seq {
    int group, first;  // its group and that one's first sequence
    int L, used;
    int off;           // pages of the sequences before it, without those that are read with their groups
    int pad;
};

struct Head {
    int magic, B, N, Hq, Hkv, D, groups, C, max_pages, num_pages;
    int blocks;
    int pad[5];
};

struct Plan {  // a plan's parts in its buffer
    Head* head;
    Cta* cta;
    Group* grp;    // [groups + 1]
    Seq* seq;      // [B + 1]
    Block* blk;    // [blocks + 1]
    Split* split;  // [C]
    Piece* piece;  // [CTA, then segment]
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
    q.grp = reinterpret_cast<Group*>(take(sizeof(Group) * ((size_t)d.groups + 1)));
    q.seq = reinterpret_cast<Seq*>(take(sizeof(Seq) * ((size_t)d.B + 1)));
    q.blk = reinterpret_cast<Block*>(take(sizeof(Block) * ((size_t)d.max_blocks() + 1)));
    q.split = reinterpret_cast<Split*>(take(sizeof(Split) * (size_t)d.C));
    q.piece = reinterpret_cast<Piece*>(take(sizeof(Piece) * (size_t)d.max_pieces()));
    if (p) *p = q;
    return n;
}

// Partial sums by rows: O [rows][D], then max [rows], then sum [rows].  The piece of
// segment s in CTA r has the rows from row0(s) + block_rows() r on: row0 counts the rows
// of the segments before s, and a segment has at most block_rows().
__host__ __device__ inline size_t partial_rows(const Dims& d) {
    return (size_t)d.B * d.N * d.Hq + (size_t)d.block_rows() * d.C;
}
__host__ __device__ inline size_t workspace_bytes(const Dims& d) { return partial_rows(d) * (d.D + 2) * sizeof(float); }
// ... with n_g sequences from seq0 on in the segment's group, whose block starts at node0.
__host__ __device__ inline int row0_of(const Dims& d, int seq0, int n_g, int g, int node0) {
    return d.G * (d.Hkv * d.N * seq0 + g * n_g * d.N + (node0 - seq0 * d.N));
}

struct Launch {
    lucetree_attn_args a;  // a.out is not used
    Dims d;
    Plan plan;
    float* ws;
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
