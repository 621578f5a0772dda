// Where a packed step's tokens belong, from the requests' lengths: token n of the
// step is token n - first[b] of request b, first the running sum of q_len; it sits
// at position total_len[b] - q_len[b] + (n - first[b]), in the cache row that the
// block table names.
//
// One launch: every block forms the running sums of all requests (up to 4,096: 16
// lengths a thread and one scan, 16 KB from L2) and its tokens look theirs up by
// bisection in shared memory. Bound by latency: the lengths, a scan, a lookup in the
// table, a store: 3.1 us for 64 requests of one token, 5.8 for 500 of up to 2,048
// (200,000 tokens, 2.5 MB; a scan by one block ahead of the rest would be a second launch).
#include <algorithm>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kSlotThreads = 256, kSlotRows = 4096, kSlotPer = kSlotRows / kSlotThreads, kSlotTokens = 4;

struct SlotParams {
  const int32_t* q_len;
  const int32_t* total_len;
  int32_t* slots;
  int32_t* positions;
  int32_t* row_of;
  int32_t* first;
  long long cap;        // tokens that a row of the cache holds
  int rows, tokens;
  Paging pg;
};

__global__ void __launch_bounds__(kSlotThreads) slot_map_kernel(const SlotParams p) {
  __shared__ int s_first[kSlotRows + 1];   // clipped to `tokens`
  __shared__ uint32_t s_tot[32];
  const int tid = threadIdx.x;
  // lengths, clipped to the step's (sums of 4,096 of them would leave 32 bits: the
  // running sums are kept in 64 and clipped again)
  int len[kSlotPer];
  long long sum = 0;
  const int per = (p.rows + kSlotThreads - 1) / kSlotThreads;
#pragma unroll
  for (int j = 0; j < kSlotPer; ++j) {
    const int b = tid * per + j;
    const int x = j < per && b < p.rows ? __ldg(p.q_len + b) : 0;
    len[j] = x < 0 ? 0 : min(x, p.tokens);
    sum += len[j];
  }
  uint32_t total;
  const uint32_t mine = static_cast<uint32_t>(sum < p.tokens ? sum : p.tokens);
  // a scan that saturates at `tokens` (below 2^31: a sum of two fits)
  const int lane = tid & 31, wid = tid >> 5;
  uint32_t x = mine;
  const uint32_t most = static_cast<uint32_t>(p.tokens);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = min(x + y, most);
  }
  if (lane == 31) s_tot[wid] = x;
  uint32_t before = __shfl_up_sync(0xffffffffu, x, 1);
  if (lane == 0) before = 0;
  __syncthreads();
  total = 0;
  for (int w = 0; w < kSlotThreads / 32; ++w) {
    if (w == wid) before = min(before + total, most);
    total = min(total + s_tot[w], most);
  }
  uint32_t at = before;
#pragma unroll
  for (int j = 0; j < kSlotPer; ++j) {
    const int b = tid * per + j;
    if (j < per && b < p.rows) s_first[b] = static_cast<int>(at);
    at = min(at + static_cast<uint32_t>(len[j]), most);
  }
  if (tid == 0) s_first[p.rows] = static_cast<int>(total);
  __syncthreads();
  if (p.first && blockIdx.x == 0)
    for (int b = tid; b <= p.rows; b += kSlotThreads) p.first[b] = s_first[b];
#pragma unroll
  for (int j = 0; j < kSlotTokens; ++j) {
    const long long n64 = (static_cast<long long>(blockIdx.x) * kSlotTokens + j) * kSlotThreads + tid;
    if (n64 >= p.tokens) break;
    const int n = static_cast<int>(n64);
    int row = -1, pos = 0, slot = -1;
    if (n < static_cast<int>(total)) {
      int lo = 0, hi = p.rows;             // the last row whose first is at most n
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_first[mid] <= n) lo = mid;
        else hi = mid;
      }
      row = lo;
      // (in 64 bits: lengths on the device may be anything)
      const long long at64 = static_cast<long long>(__ldg(p.total_len + row)) - __ldg(p.q_len + row) + (n - s_first[row]);
      pos = at64 < 0 ? 0 : at64 > 0x7fffffffLL ? 0x7fffffff : static_cast<int>(at64);
      if (at64 >= 0 && at64 < p.cap) {
        if (p.pg.table) {
          const int blk = __ldg(p.pg.table + static_cast<long long>(row) * p.pg.per_seq + (pos >> p.pg.shift));
          if (blk >= 0 && blk < p.pg.num_blocks) slot = (blk << p.pg.shift) + (pos & ((1 << p.pg.shift) - 1));
        } else {
          slot = static_cast<int>(row * p.cap + pos);
        }
      }
    }
    p.slots[n] = slot;
    if (p.positions) p.positions[n] = pos;
    if (p.row_of) p.row_of[n] = row;
  }
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int dsa_slot_map(int rows, int64_t tokens, const dsa_kv_pages* pages, int32_t cache_capacity,
                            const int32_t* q_len, const int32_t* total_len, int32_t* slots, int32_t* positions,
                            int32_t* row_of, int32_t* first, void* stream) {
  reset_launches();
  if (rows < 1 || rows > kSlotRows) return report_errorf(DSA_ERR_INVALID_ARG, "rows %d outside 1..%d", rows, kSlotRows);
  if (tokens < 0 || tokens > (1LL << 30)) return report_error(DSA_ERR_INVALID_ARG, "tokens must be 0 .. 2^30");
  SlotParams p{};
  if (pages) {
    dsa_full_problem q{};
    q.num_kv_heads = 1;
    const long long cap = static_cast<long long>(pages->block_size) * pages->blocks_per_seq;
    if (pages->block_size < 1 || pages->blocks_per_seq < 1 || cap > 0x7fffffffLL)
      return report_error(DSA_ERR_INVALID_ARG, "block_size * blocks_per_seq must lie in 1 .. 2^31 - 1");
    q.cache_capacity = static_cast<int32_t>(cap);
    if (int rc = check_full_pages(&q, pages, &p.pg)) return rc;
    p.cap = cap;
  } else {
    if (cache_capacity < 1 || static_cast<long long>(rows) * cache_capacity > 0x7fffffffLL)
      return report_error(DSA_ERR_INVALID_ARG, "without pages rows * cache_capacity must lie in 1 .. 2^31 - 1");
    p.cap = cache_capacity;
  }
  if (!q_len || !total_len || (!slots && tokens > 0))
    return report_error(DSA_ERR_INVALID_ARG, "q_len, total_len and slots are required");
  const void* arrays[] = {q_len, total_len, slots, positions, row_of, first};
  const long long bytes[] = {4LL * rows, 4LL * rows, 4 * tokens, 4 * tokens, 4 * tokens, 4LL * (rows + 1)};
  for (const void* x : arrays)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return report_error(DSA_ERR_MISALIGNED, "all arrays must be 4-byte aligned");
  const long long table_bytes = pages ? 4LL * rows * pages->blocks_per_seq : 0;
  for (int o = 2; o < 6; ++o) {
    if (!arrays[o] || !bytes[o]) continue;
    if (pages && overlap(arrays[o], bytes[o], pages->block_table, table_bytes))
      return report_error(DSA_ERR_INVALID_ARG, "a result overlaps the block table");
    for (int i = 0; i < o; ++i)
      if (arrays[i] && bytes[i] && overlap(arrays[o], bytes[o], arrays[i], bytes[i]))
        return report_error(DSA_ERR_INVALID_ARG, "a result overlaps an input or another result");
  }
  if (tokens == 0 && !first) return DSA_OK;
  int sms = 0;
  if (int rc = current_device(&sms)) return rc;
  p.q_len = q_len, p.total_len = total_len, p.slots = slots, p.positions = positions, p.row_of = row_of, p.first = first;
  p.rows = rows;
  p.tokens = static_cast<int>(tokens);
  const long long blocks = std::max<long long>(1, (tokens + kSlotThreads * kSlotTokens - 1) / (kSlotThreads * kSlotTokens));
  const cudaError_t e = launch_kernel("slot_map_kernel", slot_map_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kSlotThreads), 0,
                                      static_cast<cudaStream_t>(stream), false, p);
  if (e != cudaSuccess) return report_errorf(DSA_ERR_CUDA, "slot_map launch: %s", cudaGetErrorString(e));
  return DSA_OK;
}
