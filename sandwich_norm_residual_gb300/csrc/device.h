// What the library's translation units share of its per-device state.
#pragma once

#include "beam_boundary.h"

namespace beam {

struct Device {
    int ordinal;
    int sms;
    unsigned int* status_word;  // device address of the word that beam_sync_status reads
};

// The current device, BEAM_ERR_DEVICE when it is not an sm_103 GPU.
beam_status device(Device* out);

}  // namespace beam
