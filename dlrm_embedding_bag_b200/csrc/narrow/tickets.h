// How the CTAs of a launch take its chunks in order, from one word in memory that its user can
// write too. Written over the word's values alone, so that the rule can be checked on the CPU.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define DLRM_TICKET_FN __host__ __device__ __forceinline__
#else
#define DLRM_TICKET_FN inline
#endif

namespace dlrm {

// A CTA starts with the chunk of its own number. At its start it sees to it that the word is raised:
// where it is not, it is set to kDrawing (an exchange, if it still holds what was seen, so that
// only one CTA does; or an atomic maximum, which does as much for a word below kDrawing). Then the
// CTA adds 1 to it for each ticket (an atomic sum). So tickets, what the word is above kDrawing,
// count from 0 whatever it was left at. A CTA draws a ticket for each chunk that it works on
// (one if it has none), which is one for each chunk in all. Who draws the last one writes the
// word back to 0: all others have drawn theirs.
//
// A word that was left raised (a number from -2^31 to -2^30) is not told from one that this launch
// raised: chunks are then left out. None is taken that the launch does not have, whatever the
// word was.
constexpr uint32_t kDrawing = 1u << 31;
constexpr uint32_t kMostTickets = 1u << 30;

DLRM_TICKET_FN bool raised(uint32_t word) { return word - kDrawing <= kMostTickets; }

// The chunk to take next, of `chunks`, where the word was `drawn` before its draw and `ctas` CTAs
// started; `chunks` or above: there is none. (chunks is at most kMostTickets, ctas less than that.)
DLRM_TICKET_FN int next_chunk(uint32_t drawn, int chunks, int ctas) {
  const uint32_t ticket = drawn & ~kDrawing;
  return ticket >= static_cast<uint32_t>(chunks) ? chunks : static_cast<int>(ticket) + ctas;
}

// Whether that draw was the launch's last one.
DLRM_TICKET_FN bool last_ticket(uint32_t drawn, int chunks) {
  return drawn == kDrawing + static_cast<uint32_t>(chunks > 1 ? chunks - 1 : 0);
}

}  // namespace dlrm
